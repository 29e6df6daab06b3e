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
    if (ld < row || ld * (dtype == GDN_BF16 ? 2 : 4) % 16 != 0) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status_t check_cache(const gdn_kv_cache_t* c, gdn::CacheView* out) {
    if (!c || c->n_pages < 1 || c->Hk < 1) return GDN_ERR_INVALID_ARG;
    if (c->dtype != GDN_BF16 && c->dtype != GDN_E4M3) return GDN_ERR_INVALID_ARG;
    if (!row_dim_ok(c->D) || c->Hk > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    int shift = 0;
    while ((1 << shift) < c->page && shift < 20) ++shift;
    if (c->page < 16 || c->page > 1024 || (1 << shift) != c->page) return GDN_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return GDN_ERR_INVALID_ARG;
    if (c->dtype == GDN_E4M3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
        return GDN_ERR_INVALID_ARG;
    *out = gdn::CacheView{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, shift, c->Hk, c->D, c->dtype == GDN_E4M3};
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
    if ((q_out == q && ld_q != (int64_t)H * D) || (k_out == k && ld_k != (int64_t)Hk * D) || q_out == k_out)
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
    if (!k || !v || k == v || !aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_INVALID_ARG;
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
    if (!new_seq_lens || new_seq_lens == seq_lens || (M > 0 && !accepted)) return GDN_ERR_INVALID_ARG;
    a.path = accepted; a.M = M; a.new_lens = new_seq_lens;
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_kv_accept(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_tree_attention_workspace_size(const gdn_kv_cache_t* cache, int N, int H, int max_nodes) {
    if (!cache || N < 0 || H <= 0 || cache->Hk <= 0 || cache->Hk > kMaxHeads || H % cache->Hk != 0 ||
        H / cache->Hk > 64 || max_nodes <= 0 || max_nodes > gdn::kMaxNodes ||
        !(cache->D == 64 || cache->D == 128 || cache->D == 256))
        return 0;
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
    if (H < 1 || H % a.c.Hk != 0 || max_nodes < 1 || !(scale > 0.f) || !(scale <= 3.4e38f)) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 || max_nodes > gdn::kMaxNodes) return GDN_ERR_UNSUPPORTED;
    if (!(a.c.D == 64 || a.c.D == 128 || a.c.D == 256) || H / a.c.Hk > 64) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)N * a.c.Hk >= (int64_t)1 << 31) return GDN_ERR_UNSUPPORTED;
    if (a.c.n_pages >= ((int64_t)1 << 31) / ((int64_t)a.c.Hk << a.c.page_shift)) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (!q || !o || o == q || !aligned(q, 16) || !aligned(o, 16) || !aligned(gate, 16) || !aligned(mask, 8) ||
        !aligned(lse, 4) || (gate && gate == o))
        return GDN_ERR_INVALID_ARG;
    if (gdn_status_t st = check_stride(ld_q, H, a.c.D, dtype)) return st;
    if (!workspace || !aligned(workspace, 256) ||
        ws_bytes < gdn_tree_attention_workspace_size(cache, N, H, max_nodes))
        return GDN_ERR_WORKSPACE;
    a.q = q; a.ld_q = ld_q; a.T = T; a.H = H; a.mask = mask; a.max_nodes = max_nodes; a.scale = scale; a.gate = gate;
    a.o = o; a.lse = lse; a.workspace = workspace; a.wait_ns = gdn::wait_limit_ns();
    a.status = gdn::device_status_ptr();
    if (!a.status) return GDN_ERR_CUDA;
    return from_cuda(gdn::launch_tree_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
