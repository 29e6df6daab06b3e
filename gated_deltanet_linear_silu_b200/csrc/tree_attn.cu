// Attention of a drafted tree over the paged cache (one node: a plain decode
// step). For node i of a sequence with `base` cached tokens before the draft,
// and query head h reading key/value head h / (H / Hk):
//
//   s_j = scale q_i . k_j,   j < base, or j - base a set bit of mask_i
//   o_i = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},   m = max_j s_j
//
// times sigmoid(gate) when a gate is given; a row that sees nothing is zero
// with lse = -inf.
//
// Bound by reading the cache: 2 D bytes (e4m3; twice that in bf16) per cached
// token and head, against 4 D flops per query row.
//
// This file: up to 16 query rows of a key/value head (a decode step, a short
// draft), where the cache streams through registers. Tokens are the M side of
// mma.sync m16n8k16 and rows the N side, eight at a time, so that few rows
// waste nothing: S^T = K Q^T and O^T = V^T P^T. A warp takes 16 tokens per step
// from a private ring in shared memory that it fills with cp.async; nothing but
// the end of a segment synchronises the CTA. The order of the contraction over
// d and of the output's d is free: a lane's fragments are whole 16-byte pieces
// of a row, whatever elements those are. More rows: tree_attn_tc.cu. At the
// border, 16 rows (64 sequences of 8192 tokens, 8 key/value heads of 128, four
// nodes of four query heads), this kernel takes 241 us and the other 337 from an
// e4m3 cache, 354 and 362 from a bf16 one; one node: 200 and 327.
//
// One node there is 1.1 GB of cache in 184 to 194 us, 5.7 to 6.0 TB/s (87 to 92 %
// of a copy's rate): HBM is nearly the bound, the rest is the instructions
// between its loads. 9.3 us for one sequence of 1021 tokens are latency: bounds and
// shares 1 us, a page's id and its rows 3, the four warps' sums 1, the join 3.5.
//
// e4m3 values enter the products as f16, exactly, by the hardware conversion
// (one instruction for two; through bf16 it would take five), and so do the
// queries, each row scaled by a power of two that leaves f16 as many bits as it has
// (exact down to 2^-31 of the row's largest element, off by 2^-39 of it below). Keys' scales
// multiply the scores in fp32. Values' scales multiply the probabilities; the
// running reference R of a row is over s_j + log2 vs_j, so that the largest
// weight e^{s - R} vs is 2^7 and f16 (11 bits) holds the others next to
// it, however the scales differ. R moves, and the sums are rescaled, only when
// a weight would pass 2^15 (bf16: one, and 2^8). Sums, maxima and outputs are fp32.
// From a bf16 cache the numerators are bf16, since both operands of a product have one
// type: 8 bits, half a step of each, where fp32 ones would take three products for one.
#include <cfloat>

#include "kv_page.cuh"
#include "launch.h"
#include "tree_attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;           // most query rows of a unit
constexpr int kTile = 16 * kWarps;  // tokens of a tile: 16 per warp

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Transpose of an 8 x 8 matrix of 16-bit values, one row's pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, bool E4M3, int NT>
struct Config {
    static constexpr int kRowBytes = E4M3 ? D : 2 * D;
    static constexpr int kChunks = kRowBytes / 16;  // 16-byte pieces of a row
    static constexpr int kSide = 16 * kRowBytes;    // keys (or values) of a step
    static constexpr int kStage = 2 * kSide + (E4M3 ? 128 : 0);
    // Q fragments stay in registers while they and the output leave room
    static constexpr bool kQInSmem = NT * D > 256;
    static constexpr int kQBytes = kQInSmem ? NT * D / 16 * 256 : 0;
    static constexpr int kMerge = kWarps * 8 * NT * (D + 2) * 4;
    static constexpr int ring(int stages) { return stages * kStage * kWarps; }
    static constexpr int smem(int stages) { return (ring(stages) > kMerge ? ring(stages) : kMerge) + kQBytes; }
    static constexpr bool fits(int ctas, int stages) { return ctas * (smem(stages) + 1536) <= 227 * 1024; }
    // CTAs per SM: what the registers of the output allow, then what a ring of
    // two stages (the one in use and one in flight) allows; then stages
    static constexpr int kWant = NT * D <= 128 ? 4 : NT * D <= 256 ? 3 : 2;
    static constexpr int kCtas = fits(kWant, 2) ? kWant : fits(kWant - 1, 2) ? kWant - 1 : 1;
    static constexpr int kStages = fits(kCtas, 4) ? 4 : fits(kCtas, 3) ? 3 : 2;
    static constexpr int kSmem = smem(kStages);

    // Row of token label x (0..7) of a step's half, and the 16-byte piece that
    // lane row r takes of a value row's 128 bytes: eight lanes of a shared-memory
    // access then meet eight different bank groups under the swizzle below.
    static __device__ __forceinline__ int token(int x) { return kRowBytes >= 128 ? ((x & 1) << 2) | (x >> 1) : x; }
    static __device__ __forceinline__ int piece(int r) { return kRowBytes >= 128 ? ((r & 1) << 2) | (r >> 1) : r; }
    static __device__ __forceinline__ int offset(int row, int chunk) {
        const int swz = kRowBytes >= 128 ? row & 7 : (row >> 1) & 3;
        return row * kRowBytes + ((chunk ^ swz) << 4);
    }
};

// First of the four elements that lane column c holds for k-step ks of the
// first product (its two fragment words take two each).
template <bool E4M3>
__device__ __forceinline__ int k_elem(int ks, int c) {
    return E4M3 ? 64 * (ks >> 2) + 16 * c + 4 * (ks & 3) : 32 * (ks >> 1) + 8 * c + 4 * (ks & 1);
}

// NT: groups of eight query rows.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, (Config<D, E4M3, NT>::kCtas)) tree_kernel(TreeArgs a) {
    using C = Config<D, E4M3, NT>;
    constexpr int kSteps = D / 16, RB = C::kRowBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = a.H / a.c.Hk;
    // (in this order: the joining kernel reads the call's inputs before it waits, so
    // it may start only when what wrote them is done)
    pdl_wait_previous();
    pdl_launch_dependents();
    const Share share = find_share<kRows, kTile, kThreads>(a);

    float* partials = partial_base(a);
    uint8_t* ring = smem + warp * C::kStages * C::kStage;
    uint32_t* q_smem = reinterpret_cast<uint32_t*>(smem + C::kSmem - C::kQBytes);

    Segment seg;
    for (bool have = first_segment<kRows, kTile>(a, share, seg); have; have = next_segment<kRows, kTile>(a, share, seg)) {
        const Seq& seq = seg.seq;
        const int tile0 = seg.tile0, tile1 = seg.tile1;
        const int hk = seg.hk, rows = seg.rows;
        const int base = seq.len - seq.nodes;
        const int64_t head_rows = (int64_t)hk << a.c.page_shift;

        // ---- the ring: this warp's 16 tokens of a tile into stage st. Pages hold a
        // multiple of 16 tokens: a step lies in one, its rows back to back.
        const int32_t* table = a.p.table + (int64_t)seg.n * a.p.max_pages;
        auto page_id = [&](int tile) -> int {  // page of the step; looked at by issue(), a tile later
            const int pos = tile * kTile + warp * 16;
            return tile < tile1 && pos < seq.len ? __ldg(table + (pos >> a.c.page_shift)) : 0;
        };
        auto issue = [&](int tile, int id, int st) {
            uint8_t* dst = ring + st * C::kStage;
            if (tile < tile1) {
                const int pos = tile * kTile + warp * 16;
                int left = seq.len - pos;  // tokens that exist
                if (id < 0 || id >= a.c.n_pages) {
                    if (lane == 0) set_status(a.status, kStatusBadSeqlens);
                    left = id = 0;
                }
                const int64_t row = (((int64_t)id * a.c.Hk + hk) << a.c.page_shift) + (pos & ((1 << a.c.page_shift) - 1));
                const uint8_t* kb = static_cast<const uint8_t*>(a.c.k) + row * RB + 16 * lane;
                const uint8_t* vb = static_cast<const uint8_t*>(a.c.v) + row * RB + 16 * lane;
                if (left >= 16) {
#pragma unroll
                    for (int i = 0; i < C::kSide / 512; ++i) {
                        const int p = lane + 32 * i;
                        cp_async_16(dst + C::offset(p / C::kChunks, p % C::kChunks), kb + 512 * i);
                    }
#pragma unroll
                    for (int i = 0; i < C::kSide / 512; ++i) {
                        const int p = lane + 32 * i;
                        cp_async_16(dst + C::kSide + C::offset(p / C::kChunks, p % C::kChunks), vb + 512 * i);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < C::kSide / 512; ++i) {
                        const int p = lane + 32 * i, tok = p / C::kChunks;
                        const bool on = tok < left;
                        cp_async_zfill16(dst + C::offset(tok, p % C::kChunks), on ? kb + 512 * i : a.c.k, on);
                        cp_async_zfill16(dst + C::kSide + C::offset(tok, p % C::kChunks), on ? vb + 512 * i : a.c.v, on);
                    }
                }
                if (E4M3) {
                    const float* s = lane < 16 ? a.c.k_scale : a.c.v_scale;
                    const bool on = (lane & 15) < left;
                    cp_async_zfill4(dst + 2 * C::kSide + 4 * lane, on ? s + row + (lane & 15) : s, on);
                }
            }
            cp_async_commit_group();
        };
#pragma unroll
        for (int st = 0; st < C::kStages - 1; ++st) issue(tile0 + st, page_id(tile0 + st), st);
        int next_id = page_id(tile0 + C::kStages - 1);

        // ---- queries: row 8 g + r as this lane's fragment column; what rows
        // 8 g + 2 c + {0, 1} (this lane's scores) see of the draft
        uint32_t qf[C::kQInSmem ? 1 : NT][C::kQInSmem ? 1 : kSteps][2];
        // factor of the scores (log2 units); reference, its negative (0 while there is
        // none) and the weight (log2) that moves it; sum
        float mul[NT][2], ref[NT][2], minus[NT][2], l[NT][2];
        uint64_t sees[NT][2];
#pragma unroll
        for (int g = 0; g < NT; ++g) {
            const bool live = 8 * g + r < rows;
            const int64_t t = seq.first + (live ? 8 * g + r : 0) / G;
            const uint16_t* qp = static_cast<const uint16_t*>(a.q) + t * a.ld_q + (int64_t)(hk * G + (live ? 8 * g + r : 0) % G) * D;
            float down = 1.f, up = 1.f;  // the row's power of two (query_scale)
            if (E4M3) {
                uint32_t m = 0;
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    const uint2 x = live ? *reinterpret_cast<const uint2*>(qp + k_elem<E4M3>(ks, c)) : make_uint2(0, 0);
                    const uint32_t w[4] = {x.x & 0x7FFFu, x.x >> 16 & 0x7FFFu, x.y & 0x7FFFu, x.y >> 16 & 0x7FFFu};
                    m = max(m, max(max(w[0], w[1]), max(w[2], w[3])));
                }
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                query_scale(m, down, up);
            }
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                const uint2 x = live ? *reinterpret_cast<const uint2*>(qp + k_elem<E4M3>(ks, c)) : make_uint2(0, 0);
                uint32_t w[2] = {x.x, x.y};
                if (E4M3) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[i] = pack_f16(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
                }
                if (C::kQInSmem) {
                    if (ks % kWarps == warp)
                        *reinterpret_cast<uint2*>(q_smem + ((g * kSteps + ks) * 32 + lane) * 2) = make_uint2(w[0], w[1]);
                } else {
                    qf[C::kQInSmem ? 0 : g][C::kQInSmem ? 0 : ks][0] = w[0];
                    qf[C::kQInSmem ? 0 : g][C::kQInSmem ? 0 : ks][1] = w[1];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * g + 2 * c + i;
                mul[g][i] = __shfl_sync(0xffffffffu, up, 4 * (2 * c + i)) * a.scale * kLog2e;
                const bool on = row < rows;
                const int node = on ? row / G : 0;
                sees[g][i] = !on ? 0 : a.mask ? (uint64_t)a.mask[seq.first + node] : (2ull << node) - 1;
                // a row that is not there: a reference that no score reaches and beside which all vanish
                ref[g][i] = on ? kNegInf : 1e30f;
                minus[g][i] = on ? 0.f : -1e30f;
                l[g][i] = 0.f;
            }
        }
        if (C::kQInSmem) __syncthreads();

        float o[D / 16][NT][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int g = 0; g < NT; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][g][e] = 0.f;
        bool odd = false;  // a value of a step with drafted tokens was not finite

        int st = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            {
                int next = st + C::kStages - 1;
                if (next >= C::kStages) next -= C::kStages;
                __syncwarp();  // every lane has read the stage that is filled next
                const int id = next_id;
                next_id = page_id(tile + C::kStages);
                issue(tile + C::kStages - 1, id, next);
            }
            cp_async_wait_group<C::kStages - 1>();
            __syncwarp();  // the other lanes' copies as well
            const uint8_t* src = ring + st * C::kStage;
            if (++st == C::kStages) st = 0;
            const int pos = tile * kTile + warp * 16;
            if (pos >= seq.len) continue;

            // ---- scores: tokens label r of either half x rows 2c, 2c + 1
            float s[NT][4];
#pragma unroll
            for (int g = 0; g < NT; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[g][e] = 0.f;
#pragma unroll
            for (int j = 0; j < RB / 64; ++j) {
                uint4 kw[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    kw[h] = *reinterpret_cast<const uint4*>(src + C::offset(8 * h + C::token(r), 4 * j + c));
                constexpr int per = E4M3 ? 4 : 2;  // k-steps of a 16-byte piece
#pragma unroll
                for (int x = 0; x < per; ++x) {
                    uint32_t ka[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w[4] = {kw[h].x, kw[h].y, kw[h].z, kw[h].w};
                        if (E4M3) {
                            ka[h] = e4m3x2_to_f16x2(w[x]);
                            ka[2 + h] = e4m3x2_to_f16x2(w[x] >> 16);
                        } else {
                            ka[h] = w[(2 * x) & 3];
                            ka[2 + h] = w[(2 * x + 1) & 3];
                        }
                    }
#pragma unroll
                    for (int g = 0; g < NT; ++g) {
                        uint32_t qb[2];
                        if (C::kQInSmem) {
                            const uint2 u = *reinterpret_cast<const uint2*>(q_smem + ((g * kSteps + per * j + x) * 32 + lane) * 2);
                            qb[0] = u.x;
                            qb[1] = u.y;
                        } else {
                            qb[0] = qf[C::kQInSmem ? 0 : g][C::kQInSmem ? 0 : per * j + x][0];
                            qb[1] = qf[C::kQInSmem ? 0 : g][C::kQInSmem ? 0 : per * j + x][1];
                        }
                        mma_16816<E4M3>(s[g], ka, qb);
                    }
                }
            }
            // ---- softmax in powers of two; lv: log2 of the values' scales
            float vs[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
            float ks[2] = {1.f, 1.f};
            if (E4M3) {
                const float* sc = reinterpret_cast<const float*>(src + 2 * C::kSide);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h] = sc[8 * h + C::token(r)];
                    vs[h] = sc[16 + 8 * h + C::token(r)];
                    lv[h] = log2_scale(vs[h]);
                }
            }
            uint32_t pb[NT][2];
            const bool drafted = pos + 16 > base;  // some token is not every row's
            auto softmax = [&](auto masked_) {
                constexpr bool masked = decltype(masked_)::value;
                uint32_t on = ~0u;  // bit 4 g + e
                if (masked) {
                    on = 0;
#pragma unroll
                    for (int g = 0; g < NT; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = pos + 8 * (e >> 1) + C::token(r);
                            if (t < base || (t < seq.len && ((sees[g][e & 1] >> (t - base)) & 1))) on |= 1u << (4 * g + e);
                        }
                }
                auto seen = [&](int g, int e) { return !masked || ((on >> (4 * g + e)) & 1); };
                // s mul (+ log2 vs): largest weight of the step against the reference
                bool grown = false;
                float t[NT][4];
#pragma unroll
                for (int g = 0; g < NT; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (E4M3) s[g][e] *= ks[e >> 1];
                        t[g][e] = E4M3 ? fmaf(s[g][e], mul[g][e & 1], lv[e >> 1]) : s[g][e] * mul[g][e & 1];
                        if (!seen(g, e)) t[g][e] = kNegInf;
                        grown = grown || t[g][e] > ref[g][e & 1] + (kLazy + kLift<E4M3>);
                    }
                if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                    for (int g = 0; g < NT; ++g)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float top = fmaxf(t[g][i], t[g][2 + i]);
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            top -= kLift<E4M3>;
                            const float old = ref[g][i];
                            if (!(top > old)) continue;
                            ref[g][i] = top;
                            minus[g][i] = -top;
                            const float f = old == kNegInf ? 1.f : exp2_approx(old - top);  // nothing but zeros (or NaN) before
                            l[g][i] *= f;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                o[j][g][i] *= f;
                                o[j][g][2 + i] *= f;
                            }
                        }
                }
#pragma unroll
                for (int g = 0; g < NT; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = 2 * h + i;
                            w[i] = exp2_approx(fmaf(s[g][e], mul[g][i], minus[g][i]));
                            // a token that the row does not see adds nothing, whatever its key and scale
                            if (!seen(g, e)) w[i] = 0.f;
                            l[g][i] += w[i];
                            if (E4M3) w[i] = seen(g, e) ? w[i] * vs[h] : 0.f;
                        }
                        pb[g][h] = transpose8(E4M3 ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]));
                    }
            };
            if (drafted) softmax(Bool<true>{});
            else softmax(Bool<false>{});
            // ---- outputs: this lane's pieces of d x tokens labels 2c, 2c + 1 of either half
            const uint8_t* vsrc = src + C::kSide;
            constexpr int W = RB == 64 ? 2 : 4;   // words of a piece
            constexpr int kPieces = RB / 32 / W;  // pieces of a lane
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                uint32_t v[4][W];  // [half * 2 + token][word]
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = 8 * (x >> 1) + C::token(2 * c + (x & 1));
                    if (W == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(vsrc + C::offset(row, 8 * j + C::piece(r)));
                        v[x][0] = u.x; v[x][1] = u.y; v[x][W > 2 ? 2 : 0] = u.z; v[x][W > 3 ? 3 : 1] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(vsrc + C::offset(row, r >> 1) + 8 * (r & 1));
                        v[x][0] = u.x; v[x][1] = u.y;
                    }
                }
                if (!E4M3 && drafted) {
                    // a drafted value that is not finite must not reach the rows that do not see it:
                    // zero here, added to the others at the end of the segment (with the context's
                    // values of this step)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int w = 0; w < W; ++w) odd |= zero_non_finite(v[x][w]);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (E4M3) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {  // elements 4 w + 2 y, + 1 of the piece
                            const uint32_t sel = y ? 0x7362 : 0x5140;
                            const uint32_t h0 = __byte_perm(v[0][w], v[1][w], sel), h1 = __byte_perm(v[2][w], v[3][w], sel);
                            const uint32_t va[4] = {e4m3x2_to_f16x2(h0), e4m3x2_to_f16x2(h0 >> 16), e4m3x2_to_f16x2(h1),
                                                    e4m3x2_to_f16x2(h1 >> 16)};
#pragma unroll
                            for (int g = 0; g < NT; ++g) mma_16816<true>(o[(j * W + w) * 2 + y][g], va, pb[g]);
                        }
                    } else {
                        const uint32_t va[4] = {__byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
                                                __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632)};
#pragma unroll
                        for (int g = 0; g < NT; ++g) mma_16816<false>(o[(j * W + w) % (D / 16)][g], va, pb[g]);
                    }
                }
            }
        }
        cp_async_wait_group<0>();

        // ---- join the four warps: reference, l and o of every row
        const bool any_odd = __syncthreads_or(odd);  // and the rings are drained: they hold the sums now
        float* buf = reinterpret_cast<float*>(smem);  // [warp][row][D]
        float* mw = buf + kWarps * 8 * NT * D;        // [warp][row]
        float* lw = mw + kWarps * 8 * NT;
        constexpr int kElems = RB == 64 ? 8 : E4M3 ? 16 : 8;  // of a piece
        // Place of element d of a row: its 16 bytes exchanged within groups of eight by
        // the row, so that a warp's stores (eight pieces of four rows) meet every bank.
        auto place = [](int row, int d) {
            const int x = row >> 1 & 3;
            return (((d >> 2) ^ (kElems == 16 ? x : (x & 1) | (x & 2) << 1)) << 2) | (d & 3);
        };
#pragma unroll
        for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], 4);
                l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], 8);
                l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], 16);
                if (r == 0) {
                    mw[warp * 8 * NT + 8 * g + 2 * c + i] = ref[g][i];
                    lw[warp * 8 * NT + 8 * g + 2 * c + i] = l[g][i];
                }
            }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * g + 2 * c + i;
                float top = kNegInf;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mw[w * 8 * NT + row]);
                const float f = ref[g][i] == kNegInf ? 1.f : exp2_approx(ref[g][i] - top);
                float* y = buf + (warp * 8 * NT + row) * D;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    // output tile j: elements 2 j', 2 j' + 1 of the lane's piece j * 2 / kElems
                    const int d = (8 * (2 * j / kElems) + C::piece(r)) * kElems + 2 * j % kElems;
                    *reinterpret_cast<float2*>(y + place(row, d)) = make_float2(o[j][g][i] * f, o[j][g][2 + i] * f);
                }
            }
        __syncthreads();
        const bool whole = seg.whole();
        if (tid == 0) note_parts(a, seg);
        float* part = partials + (2 * (int)blockIdx.x + seg.later) * slot_floats(D, a.slot_rows);
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), d = 4 * (x % (D / 4));
            float mt = kNegInf, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, mw[w * 8 * NT + row]);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float m = mw[w * 8 * NT + row];
                lt += m == kNegInf ? lw[w * 8 * NT + row] : lw[w * 8 * NT + row] * exp2_approx(m - mt);
                const float4 z = *reinterpret_cast<const float4*>(buf + (w * 8 * NT + row) * D + place(row, d));
                y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
            }
            const int node = row / G, head = hk * G + row % G;
            const int64_t t = seq.first + node;
            if (!E4M3 && any_odd) {
                // values that are not finite in the steps with drafted tokens, for the rows that see
                // them: the context before the draft is every row's
                const uint64_t bits = a.mask ? (uint64_t)a.mask[t] : (2ull << node) - 1;
                const int from = max(base & ~15, tile0 * kTile), to = min(seq.len, tile1 * kTile);
                for (int p = from; p < to; ++p) {
                    if (p >= base && !((bits >> (p - base)) & 1)) continue;
                    const int64_t vr = page_row(a.p, a.c, seg.n, p);
                    if (vr < 0) continue;
                    const float4 z = load4(static_cast<const uint16_t*>(a.c.v) + (vr + head_rows) * D + d);
                    if (!(fabsf(z.x) <= FLT_MAX)) y.x += z.x;
                    if (!(fabsf(z.y) <= FLT_MAX)) y.y += z.y;
                    if (!(fabsf(z.z) <= FLT_MAX)) y.z += z.z;
                    if (!(fabsf(z.w) <= FLT_MAX)) y.w += z.w;
                }
            }
            if (!whole) {
                if (d == 0) {
                    part[row] = mt;
                    part[a.slot_rows + row] = lt;
                }
                *reinterpret_cast<float4*>(part + 2 * a.slot_rows + row * D + d) = y;
                continue;
            }
            const float inv = mt == kNegInf && lt == 0.f ? 0.f : 1.f / lt;
            y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
            const int64_t out = (t * a.H + head) * D + d;
            if (a.gate) {  // (__expf is off by 2 + 1.16 |g| ulp: 2^-17 where the sigmoid nears zero, against bf16's 2^-9)
                const float4 g = load4(static_cast<const uint16_t*>(a.gate) + out);
                y.x /= 1.f + __expf(-g.x); y.y /= 1.f + __expf(-g.y);
                y.z /= 1.f + __expf(-g.z); y.w /= 1.f + __expf(-g.w);
            }
            store4(static_cast<uint16_t*>(a.o) + out, y);
            if (a.lse && d == 0) a.lse[t * a.H + head] = mt == kNegInf && lt == 0.f ? kNegInf : mt * kLn2 + logf(lt);
        }
        __syncthreads();  // the rings are filled again
    }
}

// Joins the partials of the units that span CTAs: a warp per row, or SPLIT warps,
// a stretch of the partials each.
template <int D, int ROWS, int TN, int SPLIT>
__global__ void __launch_bounds__(SPLIT > 1 ? 32 * SPLIT : kThreads) join_kernel(TreeArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = blockIdx.x / a.c.Hk, hk = blockIdx.x % a.c.Hk;
    const int G = a.H / a.c.Hk;
    const int x = SPLIT > 1 ? blockIdx.y : blockIdx.y * kWarps + warp;  // row of the (sequence, head)
    const int rt = x / ROWS, row = x % ROWS;
    pdl_launch_dependents();
    // (inputs of the call: complete before the kernel before let this one start)
    const Seq seq = load_seq(a, n);
    const bool live = x < seq.nodes * G;
    const int64_t t = seq.first + x / G;
    const int head = hk * G + x % G;
    constexpr int V = D / 128 > 0 ? D / 128 : 1;  // float4s of a lane
    float4 gate[V];
    if (a.gate && live) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (4 * lane + 128 * v < D)
                gate[v] = load4(static_cast<const uint16_t*>(a.gate) + (t * a.H + head) * D + 4 * lane + 128 * v);
    }
    pdl_wait_previous();  // (every warp: what follows this kernel counts on the one before it being done)
    if (!live) return;
    const UnitParts parts = *unit_parts(a, rt, n, hk);
    const int c0 = parts.first >> 1;
    // one CTA had the whole unit and wrote it (or the kernel before gave up: then these are anything)
    if (parts.first < 0 || parts.last <= c0 || parts.last >= a.grid) return;
    const int all = parts.last - c0 + 1, from = SPLIT > 1 ? all * warp / SPLIT : 0;
    const int count = SPLIT > 1 ? all * (warp + 1) / SPLIT - from : all;  // of this warp
    const float* partials = partial_base(a);
    auto part = [&](int i) {
        return partials + (from + i == 0 ? parts.first : 2 * (c0 + from + i)) * slot_floats(D, a.slot_rows);
    };
    // Parts whose rows are requested together. Where units have few of them, more only
    // take registers (8 x 32768 tokens, 64 nodes: 294 us with 8 of d = 128, 301 with 16).
    constexpr int kAhead = (SPLIT > 1 ? 16 : 8) / V;
    auto load = [&](int i0, float4 (&z)[kAhead][V]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                z[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + i < count && 4 * lane + 128 * v < D)
                    z[i][v] = *reinterpret_cast<const float4*>(part(i0 + i) + 2 * a.slot_rows + row * D + 4 * lane + 128 * v);
            }
    };
    float4 z[kAhead][V], y[V];
    load(0, z);  // beside the references and sums
    float mt = kNegInf, lt = 0.f, m0 = kNegInf, l0 = 0.f;
    for (int b = 0; b < count; b += 32)
        if (b + lane < count) {
            const float* p = part(b + lane);
            const float m = p[row];
            if (b == 0) m0 = m, l0 = p[a.slot_rows + row];
            mt = fmaxf(mt, m);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < count; b += 32) {
        float f = 0.f;
        if (b + lane < count) {
            const float* p = part(b + lane);
            const float m = b == 0 ? m0 : p[row];
            f = m == kNegInf ? 1.f : exp2_approx(m - mt);  // a part that saw nothing holds zeros (or NaN)
            lt += (b == 0 ? l0 : p[a.slot_rows + row]) * f;
        }
        for (int i = 0; i < 32 && b + i < count; i += kAhead) {
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const float fi = __shfl_sync(0xffffffffu, f, (i + e) & 31);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    y[v].x = fmaf(z[e][v].x, fi, y[v].x); y[v].y = fmaf(z[e][v].y, fi, y[v].y);
                    y[v].z = fmaf(z[e][v].z, fi, y[v].z); y[v].w = fmaf(z[e][v].w, fi, y[v].w);
                }
            }
            if (b + i + kAhead < count) load(b + i + kAhead, z);
        }
    }
    lt = warp_sum(lt);
    if constexpr (SPLIT > 1) {  // the stretches, in order
        __shared__ float4 sums[SPLIT][D / 4];
        __shared__ float tops[SPLIT], totals[SPLIT];
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (4 * lane + 128 * v < D) sums[warp][lane + 32 * v] = y[v];
        if (lane == 0) {
            tops[warp] = mt;
            totals[warp] = lt;
        }
        __syncthreads();
        if (warp > 0) return;
        mt = kNegInf;
#pragma unroll
        for (int w = 0; w < SPLIT; ++w) mt = fmaxf(mt, tops[w]);
        lt = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < SPLIT; ++w) {
            const float f = tops[w] == kNegInf ? 1.f : exp2_approx(tops[w] - mt);
            lt = fmaf(totals[w], f, lt);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (4 * lane + 128 * v >= D) continue;
                const float4 u = sums[w][lane + 32 * v];
                y[v].x = fmaf(u.x, f, y[v].x); y[v].y = fmaf(u.y, f, y[v].y);
                y[v].z = fmaf(u.z, f, y[v].z); y[v].w = fmaf(u.w, f, y[v].w);
            }
        }
    }
    const bool empty = mt == kNegInf && lt == 0.f;
    const float inv = empty ? 0.f : 1.f / lt;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int d = 4 * lane + 128 * v;
        if (d >= D) continue;
        const int64_t out = (t * a.H + head) * D + d;
        float4 z = make_float4(y[v].x * inv, y[v].y * inv, y[v].z * inv, y[v].w * inv);
        if (a.gate) {
            const float4 g = gate[v];
            z.x /= 1.f + __expf(-g.x); z.y /= 1.f + __expf(-g.y);
            z.z /= 1.f + __expf(-g.z); z.w /= 1.f + __expf(-g.w);
        }
        store4(static_cast<uint16_t*>(a.o) + out, z);
    }
    if (a.lse && lane == 0) a.lse[t * a.H + head] = empty ? kNegInf : mt * kLn2 + logf(lt);
}

template <int D>
int ctas_dim(int e4m3, int rows) {
    if (rows <= 8) return e4m3 ? Config<D, true, 1>::kCtas : Config<D, false, 1>::kCtas;
    return e4m3 ? Config<D, true, 2>::kCtas : Config<D, false, 2>::kCtas;
}

// The launch's shape from its sizes alone.
struct Plan {
    bool tc;  // the tcgen05 kernel
    int grid, row_tiles, slot_rows;
};
Plan make_plan(int H, int Hk, int D, int max_nodes, int e4m3) {
    Plan p;
    const int rows = max_nodes * (H / Hk);
    p.tc = rows > kRows;
    const int tile = p.tc ? kTcRows : kRows;
    p.row_tiles = (rows + tile - 1) / tile;
    p.slot_rows = ((rows < tile ? rows : tile) + 3) / 4 * 4;
    p.grid = sm_count();
    if (!p.tc) p.grid *= D == 64 ? ctas_dim<64>(e4m3, rows) : D == 128 ? ctas_dim<128>(e4m3, rows) : ctas_dim<256>(e4m3, rows);
    if (p.grid < p.row_tiles) p.grid = p.row_tiles;  // (every row tile has a CTA)
    return p;
}

template <int D, bool E4M3, int NT>
cudaError_t launch_mma(const TreeArgs& a, cudaStream_t s) {
    using C = Config<D, E4M3, NT>;
    cudaError_t e = cudaFuncSetAttribute(tree_kernel<D, E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_kernel<D, E4M3, NT>, dim3(a.grid), dim3(kThreads), C::kSmem, s, a);
}

template <int D, bool E4M3>
cudaError_t launch_config(const TreeArgs& a, bool tc, cudaStream_t s) {
    const int rows = a.max_nodes * (a.H / a.c.Hk);
    const cudaError_t e = tc ? launch_tree_tc(a, s) : rows <= 8 ? launch_mma<D, E4M3, 1>(a, s) : launch_mma<D, E4M3, 2>(a, s);
    if (e != cudaSuccess) return e;
    // Few long units have many partials each, and few rows to share them: eight warps
    // to a row then. One sequence, one node, 2 heads of 256, with a warp and with eight: 16
    // partials 10.6 and 9.8 us, 32 partials 10.8 and 9.3, 222 (30000 tokens) 34.3 and 18.6.
    if (a.grid > (int64_t)12 * a.row_tiles * a.p.N * a.c.Hk) {
        constexpr int kSplit = 8;
        const dim3 join(a.p.N * a.c.Hk, rows);
        if (tc) return launch_pdl(join_kernel<D, kTcRows, kTcTile, kSplit>, join, dim3(32 * kSplit), 0, s, a);
        return launch_pdl(join_kernel<D, kRows, kTile, kSplit>, join, dim3(32 * kSplit), 0, s, a);
    }
    const dim3 join(a.p.N * a.c.Hk, (rows + kWarps - 1) / kWarps);
    if (tc) return launch_pdl(join_kernel<D, kTcRows, kTcTile, 1>, join, dim3(kThreads), 0, s, a);
    return launch_pdl(join_kernel<D, kRows, kTile, 1>, join, dim3(kThreads), 0, s, a);
}

template <int D>
cudaError_t launch_dim(const TreeArgs& a, bool tc, cudaStream_t s) {
    return a.c.e4m3 ? launch_config<D, true>(a, tc, s) : launch_config<D, false>(a, tc, s);
}

}  // namespace

size_t tree_workspace_bytes(int N, int H, int Hk, int D, int max_nodes, int e4m3) {
    const Plan p = make_plan(H, Hk, D, max_nodes, e4m3);
    return units_bytes(p.row_tiles, N, Hk) + 2 * (size_t)p.grid * slot_floats(D, p.slot_rows) * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeArgs& args, cudaStream_t s) {
    TreeArgs a = args;
    const Plan p = make_plan(a.H, a.c.Hk, a.c.D, a.max_nodes, a.c.e4m3);
    // no more CTAs than the tables have room for tiles
    const int64_t tiles = ((((int64_t)a.p.max_pages << a.c.page_shift) + kTile - 1) / kTile) * a.p.N * a.c.Hk * p.row_tiles;
    a.grid = tiles < p.grid ? (int)tiles : p.grid;
    if (a.grid < p.row_tiles) a.grid = p.row_tiles;
    a.row_tiles = p.row_tiles;
    a.slot_rows = p.slot_rows;
    return a.c.D == 64 ? launch_dim<64>(a, p.tc, s) : a.c.D == 128 ? launch_dim<128>(a, p.tc, s) : launch_dim<256>(a, p.tc, s);
}

}  // namespace gdn
