// C ABI of the softmax-attention layer's calls (declared in include/gdn.h):
// argument validation on the host and dispatch. No allocation, no host sync.
#include <atomic>

#include "../../include/gdn.h"
#include "attn.h"
#include "launch.h"

namespace gdn {

namespace {
constexpr int kMaxDevices = 64;
}

int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return sms;
    if (const int n = known[dev].load(std::memory_order_relaxed)) return n;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace gdn

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool act_ok(gdn_dtype_t t) { return t == GDN_F32 || t == GDN_BF16; }
gdn_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// A head of a row: a multiple of 16 elements, up to 256 (16 lanes of sixteen).
bool row_dim_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }

// Heads of a token: the kernels count its elements, and the rows of a page, in 32 bits.
constexpr int kMaxHeads = 1 << 16;

// Token stride of a [T, heads, D] tensor whose rows are dense; 0: dense.
gdn_status_t check_stride(int64_t& ld, int heads, int D, gdn_dtype_t dtype) {
    const int64_t row = (int64_t)heads * D;
    if (ld == 0) ld = row;
    if (ld < row || ld > (int64_t)1 << 56 || ld * (dtype == GDN_BF16 ? 2 : 4) % 16 != 0) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Bytes [first, first + row) of each of `rows` rows, `stride` bytes apart.
struct Span {
    const void* first;
    int64_t row, stride = 0, rows = 1;
};
Span dense(const void* p, int64_t bytes) { return {p, bytes}; }
Span tokens(const void* p, int64_t T, int heads, int D, int64_t ld, gdn_dtype_t dtype) {
    const int64_t b = dtype == GDN_BF16 ? 2 : 4;
    return {p, (int64_t)heads * D * b, ld * b, T};
}
// Whether the dense span `out` shares a byte with `in`: the first of in's rows that
// ends behind out's start begins before out's end.
bool overlap(const Span& out, const Span& in) {
    if (!out.first || !in.first || out.row <= 0 || in.row <= 0 || in.rows <= 0) return false;
    const int64_t a = (int64_t)(reinterpret_cast<uintptr_t>(out.first) - reinterpret_cast<uintptr_t>(in.first));
    const int64_t past = a - in.row;  // in's row at offset x is over before out if x <= past
    const int64_t i = past < 0 ? 0 : in.rows == 1 ? 1 : past / in.stride + 1;
    return i < in.rows && i * in.stride < a + out.row;
}
template <typename... Ins>
bool overlaps(const Span& out, const Ins&... ins) {
    return (overlap(out, ins) || ...);
}
// Of a cache: its keys, values and their scales (0 to 3).
Span cache_part(const gdn::CacheView& c, int part) {
    const void* const p[4] = {c.k, c.v, c.e4m3 ? c.k_scale : nullptr, c.e4m3 ? c.v_scale : nullptr};
    const __int128 bytes = (__int128)c.n_pages * c.Hk * (part > 1 ? 4 : c.e4m3 ? c.D : 2 * c.D) << c.page_shift;
    const int64_t most = (int64_t)1 << 60;  // (more than any address space: a + row stays in 64 bits)
    return dense(p[part], bytes < most ? (int64_t)bytes : most);
}
bool overlaps_cache(const Span& out, const gdn::CacheView& c) {
    return overlaps(out, cache_part(c, 0), cache_part(c, 1), cache_part(c, 2), cache_part(c, 3));
}
// For calls that write the cache: whether a part lies on another or on an input.
template <typename... Ins>
bool cache_overlaps(const gdn::CacheView& c, const Ins&... ins) {
    for (int x = 0; x < 4; ++x) {
        for (int y = 0; y < x; ++y)
            if (overlap(cache_part(c, x), cache_part(c, y))) return true;
        if (overlaps(cache_part(c, x), ins...)) return true;
    }
    return false;
}
Span table_of(const gdn::PageArgs& p) { return dense(p.table, (int64_t)4 * p.N * p.max_pages); }
Span lens_of(const gdn::PageArgs& p) { return dense(p.lens, (int64_t)4 * p.N); }
Span cu_of(const gdn::PageArgs& p) { return dense(p.cu, (int64_t)4 * (p.N + 1)); }
bool overlaps_pages(const Span& out, const gdn::PageArgs& p) { return overlaps(out, table_of(p), lens_of(p), cu_of(p)); }

// What a cache's fields say without its memory; log2 of the page's tokens.
gdn_status_t check_cache_shape(const gdn_kv_cache_t* c, int* page_shift) {
    if (!c || c->n_pages < 1 || c->Hk < 1) return GDN_ERR_INVALID_ARG;
    if (c->dtype != GDN_BF16 && c->dtype != GDN_E4M3) return GDN_ERR_INVALID_ARG;
    if (!row_dim_ok(c->D) || c->Hk > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    int shift = 0;
    while ((1 << shift) < c->page && shift < 20) ++shift;
    if (c->page < 16 || c->page > 1024 || (1 << shift) != c->page) return GDN_ERR_UNSUPPORTED;
    *page_shift = shift;
    return GDN_OK;
}

gdn_status_t check_cache(const gdn_kv_cache_t* c, gdn::CacheView* out) {
    int shift = 0;
    if (gdn_status_t st = check_cache_shape(c, &shift)) return st;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return GDN_ERR_INVALID_ARG;
    if (c->dtype == GDN_E4M3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
        return GDN_ERR_INVALID_ARG;
    *out = gdn::CacheView{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, shift, c->Hk, c->D, c->dtype == GDN_E4M3};
    return GDN_OK;
}

// The tree attention's sizes, for a cache that check_cache_shape allows.
gdn_status_t check_tree(const gdn_kv_cache_t* c, int page_shift, int N, int H, int max_nodes) {
    if (N < 0 || H < 1 || H % c->Hk != 0 || max_nodes < 1) return GDN_ERR_INVALID_ARG;
    if (max_nodes > gdn::kMaxNodes || H / c->Hk > 64) return GDN_ERR_UNSUPPORTED;
    if (!(c->D == 64 || c->D == 128 || c->D == 256)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)N * c->Hk >= (int64_t)1 << 31) return GDN_ERR_UNSUPPORTED;
    if (c->n_pages >= ((int64_t)1 << 31) / ((int64_t)c->Hk << page_shift)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status_t check_pages(const int32_t* table, int max_pages, const int32_t* lens, const int32_t* cu, int N, int64_t T,
                         gdn::PageArgs* out) {
    if (N < 0 || T < 0 || max_pages < 0 || (N == 0 && T > 0)) return GDN_ERR_INVALID_ARG;
    if (T >= (int64_t)1 << 31) return GDN_ERR_UNSUPPORTED;  // cu_seqlens is int32
    if (N > 0 && (!table || !lens || !cu || max_pages < 1)) return GDN_ERR_INVALID_ARG;
    *out = gdn::PageArgs{table, lens, cu, N, max_pages};
    return GDN_OK;
}

gdn_status_t check_norm(int H, int Hk, int D, const float* q_w, const float* k_w, float eps, const int32_t* pos,
                        const double* inv_freq, int rotary, int interleaved) {
    if (H < 1 || Hk < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return GDN_ERR_INVALID_ARG;
    if (!row_dim_ok(D) || H > kMaxHeads || Hk > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    if (rotary < 0 || rotary > D) return GDN_ERR_INVALID_ARG;
    if (rotary % 16 != 0) return GDN_ERR_UNSUPPORTED;
    if (!aligned(q_w, 16) || !aligned(k_w, 16)) return GDN_ERR_INVALID_ARG;
    if (!q_w || !k_w || !pos || (rotary > 0 && !inv_freq)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_qk_norm_rope(const void* q, const void* k, gdn_dtype_t dtype, int64_t T, int H, int Hk, int D,
                              int64_t ld_q, int64_t ld_k, const float* q_w, const float* k_w, float eps,
                              const int32_t* positions, const double* inv_freq, int rotary, int interleaved,
                              void* q_out, void* k_out, void* stream) {
    if (!act_ok(dtype) || T < 0) return GDN_ERR_INVALID_ARG;
    if (T >= (int64_t)1 << 31) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (gdn_status_t st = check_norm(H, Hk, D, q_w, k_w, eps, positions, inv_freq, rotary, interleaved)) return st;
    if (!q || !k || !q_out || !k_out) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16)) return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_stride(ld_q, H, D, dtype)) return st;
    if (gdn_status_t st = check_stride(ld_k, Hk, D, dtype)) return st;
    // in place is row by row: only over dense rows do output rows coincide with input rows
    if ((q_out == q && ld_q != (int64_t)H * D) || (k_out == k && ld_k != (int64_t)Hk * D)) return GDN_ERR_INVALID_ARG;
    // rows are read and written by different warps: otherwise nothing may lie on what is read or written
    const Span qs = tokens(q, T, H, D, ld_q, dtype), ks = tokens(k, T, Hk, D, ld_k, dtype);
    const Span qo = tokens(q_out, T, H, D, (int64_t)H * D, dtype), ko = tokens(k_out, T, Hk, D, (int64_t)Hk * D, dtype);
    const Span qw = dense(q_w, 4 * D), kw = dense(k_w, 4 * D), ps = dense(positions, 4 * T), fs = dense(inv_freq, 4 * rotary);
    const Span out_q = dense(q_out, qo.row * T), out_k = dense(k_out, ko.row * T);
    if ((q_out != q && overlap(out_q, qs)) || (k_out != k && overlap(out_k, ks)) || overlaps(out_q, ks, ko, qw, kw, ps, fs) ||
        overlaps(out_k, qs, qw, kw, ps, fs))
        return GDN_ERR_INVALID_ARG;
    gdn::RowsArgs a{};
    a.q = q; a.k = k; a.ld_q = ld_q; a.ld_k = ld_k; a.is_bf16 = dtype == GDN_BF16; a.T = T; a.H = H; a.Hk = Hk;
    a.D = D; a.q_w = q_w; a.k_w = k_w; a.eps = eps; a.pos = positions; a.inv_freq = inv_freq; a.rotary = rotary;
    a.interleaved = interleaved; a.q_out = q_out; a.k_out = k_out;
    return from_cuda(gdn::launch_rows(a, gdn::kNormRope, static_cast<cudaStream_t>(stream)));
}

gdn_status_t gdn_qk_norm_rope_cache(const void* q, const void* k, const void* v, gdn_dtype_t dtype, int64_t T, int H,
                                    int64_t ld_q, int64_t ld_k, int64_t ld_v, const float* q_w, const float* k_w,
                                    float eps, const int32_t* positions, const double* inv_freq, int rotary,
                                    int interleaved, const gdn_kv_cache_t* cache, const int32_t* page_table,
                                    int max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens, int N,
                                    void* q_out, void* stream) {
    if (!act_ok(dtype)) return GDN_ERR_INVALID_ARG;
    gdn::RowsArgs a{};
    if (gdn_status_t st = check_cache(cache, &a.c)) return st;
    if (gdn_status_t st = check_pages(page_table, max_pages, seq_lens, cu_seqlens, N, T, &a.p)) return st;
    if (T == 0) return GDN_OK;
    if (gdn_status_t st = check_norm(H, a.c.Hk, a.c.D, q_w, k_w, eps, positions, inv_freq, rotary, interleaved))
        return st;
    if (!q || !k || !v || !q_out) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16)) return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_stride(ld_q, H, a.c.D, dtype)) return st;
    if (gdn_status_t st = check_stride(ld_k, a.c.Hk, a.c.D, dtype)) return st;
    if (gdn_status_t st = check_stride(ld_v, a.c.Hk, a.c.D, dtype)) return st;
    if (q_out == q && ld_q != (int64_t)H * a.c.D) return GDN_ERR_INVALID_ARG;
    const Span qs = tokens(q, T, H, a.c.D, ld_q, dtype), ks = tokens(k, T, a.c.Hk, a.c.D, ld_k, dtype),
               vs = tokens(v, T, a.c.Hk, a.c.D, ld_v, dtype), out = dense(q_out, qs.row * T);
    const Span qw = dense(q_w, 4 * a.c.D), kw = dense(k_w, 4 * a.c.D), ps = dense(positions, 4 * T),
               fs = dense(inv_freq, 4 * rotary);
    if ((q_out != q && overlap(out, qs)) || overlaps(out, ks, vs, qw, kw, ps, fs) || overlaps_cache(out, a.c) ||
        overlaps_pages(out, a.p) || cache_overlaps(a.c, qs, ks, vs, qw, kw, ps, fs, table_of(a.p), lens_of(a.p), cu_of(a.p)))
        return GDN_ERR_INVALID_ARG;
    a.q = q; a.k = k; a.v = v; a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v; a.is_bf16 = dtype == GDN_BF16; a.T = T;
    a.H = H; a.Hk = a.c.Hk; a.D = a.c.D; a.q_w = q_w; a.k_w = k_w; a.eps = eps; a.pos = positions;
    a.inv_freq = inv_freq; a.rotary = rotary; a.interleaved = interleaved; a.q_out = q_out;
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_rows(a, gdn::kNormRopeCache, static_cast<cudaStream_t>(stream)));
}

gdn_status_t gdn_kv_write(const void* k, const void* v, gdn_dtype_t dtype, int64_t T, int64_t ld_k, int64_t ld_v,
                          const gdn_kv_cache_t* cache, const int32_t* page_table, int max_pages,
                          const int32_t* seq_lens, const int32_t* cu_seqlens, int N, void* stream) {
    if (!act_ok(dtype)) return GDN_ERR_INVALID_ARG;
    gdn::RowsArgs a{};
    if (gdn_status_t st = check_cache(cache, &a.c)) return st;
    if (gdn_status_t st = check_pages(page_table, max_pages, seq_lens, cu_seqlens, N, T, &a.p)) return st;
    if (T == 0) return GDN_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_stride(ld_k, a.c.Hk, a.c.D, dtype)) return st;
    if (gdn_status_t st = check_stride(ld_v, a.c.Hk, a.c.D, dtype)) return st;
    if (cache_overlaps(a.c, tokens(k, T, a.c.Hk, a.c.D, ld_k, dtype), tokens(v, T, a.c.Hk, a.c.D, ld_v, dtype),
                       table_of(a.p), lens_of(a.p), cu_of(a.p)))
        return GDN_ERR_INVALID_ARG;
    a.k = k; a.v = v; a.ld_k = ld_k; a.ld_v = ld_v; a.is_bf16 = dtype == GDN_BF16; a.T = T; a.Hk = a.c.Hk;
    a.D = a.c.D;
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_rows(a, gdn::kCacheWrite, static_cast<cudaStream_t>(stream)));
}

gdn_status_t gdn_kv_read(const gdn_kv_cache_t* cache, const int32_t* page_table, int max_pages,
                         const int32_t* seq_lens, const int32_t* cu_seqlens, int N, int64_t T, gdn_dtype_t dtype,
                         void* k, void* v, void* stream) {
    if (!act_ok(dtype)) return GDN_ERR_INVALID_ARG;
    gdn::ReadArgs a{};
    if (gdn_status_t st = check_cache(cache, &a.c)) return st;
    if (gdn_status_t st = check_pages(page_table, max_pages, seq_lens, cu_seqlens, N, T, &a.p)) return st;
    if (T == 0) return GDN_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_INVALID_ARG;
    const int64_t bytes = T * a.c.Hk * a.c.D * (dtype == GDN_BF16 ? 2 : 4);
    const Span ks = dense(k, bytes), vs = dense(v, bytes);
    if (overlap(ks, vs) || overlaps_cache(ks, a.c) || overlaps_cache(vs, a.c) || overlaps_pages(ks, a.p) ||
        overlaps_pages(vs, a.p))
        return GDN_ERR_INVALID_ARG;
    a.T = T; a.k = k; a.v = v; a.out_bf16 = dtype == GDN_BF16;
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_kv_read(a, static_cast<cudaStream_t>(stream)));
}

gdn_status_t gdn_kv_accept(const gdn_kv_cache_t* cache, const int32_t* page_table, int max_pages,
                           const int32_t* seq_lens, const int32_t* cu_seqlens, int N, const int32_t* accepted, int M,
                           int32_t* new_seq_lens, void* stream) {
    gdn::AcceptArgs a{};
    if (gdn_status_t st = check_cache(cache, &a.c)) return st;
    if (gdn_status_t st = check_pages(page_table, max_pages, seq_lens, cu_seqlens, N, 0, &a.p)) return st;
    if (M < 0) return GDN_ERR_INVALID_ARG;
    if (M > gdn::kMaxNodes) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    if (!new_seq_lens || (M > 0 && !accepted)) return GDN_ERR_INVALID_ARG;
    const Span out = dense(new_seq_lens, (int64_t)4 * N);  // (a sequence reads its bounds while another writes its length)
    const Span paths = dense(accepted, (int64_t)4 * N * M);
    if (overlaps_pages(out, a.p) || overlap(out, paths) || overlaps_cache(out, a.c) ||
        cache_overlaps(a.c, paths, table_of(a.p), lens_of(a.p), cu_of(a.p)))
        return GDN_ERR_INVALID_ARG;
    a.path = accepted; a.M = M; a.new_lens = new_seq_lens;
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_kv_accept(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_tree_attention_workspace_size(const gdn_kv_cache_t* cache, int N, int H, int max_nodes) {
    int shift = 0;
    if (check_cache_shape(cache, &shift) != GDN_OK || check_tree(cache, shift, N, H, max_nodes) != GDN_OK) return 0;
    const size_t b = gdn::tree_workspace_bytes(N, H, cache->Hk, cache->D, max_nodes, cache->dtype == GDN_E4M3);
    return (b + 255) / 256 * 256;
}

gdn_status_t gdn_tree_attention(const void* q, gdn_dtype_t dtype, int64_t T, int64_t ld_q, int H,
                                const gdn_kv_cache_t* cache, const int32_t* page_table, int max_pages,
                                const int32_t* seq_lens, const int32_t* cu_seqlens, int N, const int64_t* mask,
                                int max_nodes, float scale, const void* gate, void* o, float* lse, void* workspace,
                                size_t ws_bytes, void* stream) {
    if (!act_ok(dtype)) return GDN_ERR_INVALID_ARG;
    gdn::TreeArgs a{};
    if (gdn_status_t st = check_cache(cache, &a.c)) return st;
    if (gdn_status_t st = check_pages(page_table, max_pages, seq_lens, cu_seqlens, N, T, &a.p)) return st;
    if (!(scale > 0.f) || !(scale <= 3.4e38f)) return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_tree(cache, a.c.page_shift, N, H, max_nodes)) return st;
    if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(gate, 16) || !aligned(mask, 8) || !aligned(lse, 4))
        return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_stride(ld_q, H, a.c.D, dtype)) return st;
    const Span qs = tokens(q, T, H, a.c.D, ld_q, dtype), gs = dense(gate, qs.row * T), ms = dense(mask, 8 * T),
               os = dense(o, qs.row * T), ls = dense(lse, (int64_t)4 * T * H);
    for (const Span& out : {os, ls})
        if (overlaps(out, qs, gs, ms) || overlaps_cache(out, a.c) || overlaps_pages(out, a.p)) return GDN_ERR_INVALID_ARG;
    if (overlap(ls, os)) return GDN_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        ws_bytes < gdn_tree_attention_workspace_size(cache, N, H, max_nodes))
        return GDN_ERR_WORKSPACE;
    const Span ws = dense(workspace, (int64_t)gdn_tree_attention_workspace_size(cache, N, H, max_nodes));
    if (overlaps(ws, qs, gs, ms, os, ls) || overlaps_cache(ws, a.c) || overlaps_pages(ws, a.p)) return GDN_ERR_INVALID_ARG;
    a.q = q; a.ld_q = ld_q; a.T = T; a.H = H; a.mask = mask; a.max_nodes = max_nodes; a.scale = scale; a.gate = gate;
    a.o = o; a.lse = lse; a.workspace = workspace; a.wait_ns = gdn::wait_limit_ns();
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_tree_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
