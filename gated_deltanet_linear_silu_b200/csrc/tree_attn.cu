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
// token and head, against 4 D flops per query row. Rows of one key/value head
// (nodes x H / Hk) are taken 16 at a time as the M side of mma.sync m16n8k16,
// so each cached element is converted once per 16 rows. A warp streams 16
// tokens per step through a private ring in shared memory filled by
// cp.async: each lane copies exactly the 16-byte pieces that it will use as
// its fragments (the contraction order over d, and the column order of the
// output, are free, so a lane's fragments are contiguous pieces of a row), and
// the ring needs no barrier. The work -- 64-token tiles of all (sequence, kv
// head, row tile) units in one line -- is cut into equal shares, one per CTA,
// so that ragged lengths and few sequences load every SM alike; a unit that
// spans CTAs leaves partial sums (m, l, o unnormalised, fp32) in the workspace,
// which a second kernel joins.
//
// e4m3 values enter the products as bf16, exactly (a bit rearrangement times
// 2^120); keys' scales multiply the scores and values' scales the
// probabilities, both fp32. The probabilities are rounded to bf16 for the
// second product (at most 2^-8 relative each, with errors that average out over
// the sum); sums, maxima and outputs are fp32.
#include <cfloat>
#include <climits>

#include "kv_page.cuh"
#include "launch.h"
#include "tree_attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;           // query rows of a unit
constexpr int kTile = 16 * kWarps;  // tokens of a tile: 16 per warp
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool E4M3>
struct Config {
    static constexpr int kElem = E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;
    static constexpr int kKChunks = kRowBytes / 64;                     // 16-byte pieces of a key row per lane (4 lanes)
    static constexpr int kVBytes = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;  // piece of a value row (8 lanes)
    static constexpr int kVChunks = kRowBytes / 8 / kVBytes;
    static constexpr int kVElems = kVBytes / kElem;
    static constexpr int kKStage = 2 * kKChunks * 512;                  // 16 tokens of one warp
    static constexpr int kVStage = 4 * kVChunks * kVBytes * 32;
    static constexpr int kScales = E4M3 ? 128 : 0;                      // k then v scales of 16 tokens
    static constexpr int kStage = kKStage + kVStage + kScales;
    // stages: about 8 KB per warp and stage at two or three CTAs per SM fill the
    // SM's share of bandwidth times latency several times over
    static constexpr int kStages = kStage > 8000 ? 3 : 4;
    static constexpr int kRing = kStages * kStage * kWarps;
    static constexpr int kMerge = kWarps * kRows * D * 4 + kWarps * kRows * 8;
    static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + (D == 256 ? D / 16 * 512 : 0);
    static constexpr int kCtas = kSmem > 113 * 1024 ? 1 : kSmem > 75 * 1024 ? 2 : 3;
};

// The fragments' element order: k-step ks of the first product takes, from
// lane column c, elements dk .. dk + 3 of the row; word 0 of the fragment pair
// holds elements {0, 2} (e4m3: even bytes) or {0, 1} (bf16), word 1 the others.
template <bool E4M3>
__device__ __forceinline__ int k_elem(int ks, int c) {
    return E4M3 ? 64 * (ks >> 2) + 16 * c + 4 * (ks & 3) : 32 * (ks >> 1) + 8 * c + 4 * (ks & 1);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, (Config<D, E4M3>::kCtas)) tree_kernel(TreeArgs a) {
    using C = Config<D, E4M3>;
    constexpr int kSteps = D / 16;
    constexpr bool kQInSmem = D == 256;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = a.H / a.c.Hk;
    pdl_launch_dependents();

    const Share share = find_share<kRows, kTile, kThreads>(a);

    float* partials = partial_base(a);
    uint8_t* ring = smem + warp * C::kStages * C::kStage;
    uint32_t* q_smem = reinterpret_cast<uint32_t*>(smem + C::kSmem - (kQInSmem ? kSteps * 512 : 0));

    Segment seg;
    for (bool have = first_segment<kRows, kTile>(a, share, seg); have; have = next_segment<kRows, kTile>(a, share, seg)) {
        const Seq& seq = seg.seq;
        const int tile0 = seg.tile0, tile1 = seg.tile1;
        const int hk = seg.hk, rt = seg.rt, rows = seg.rows;
        const int base = seq.len - seq.nodes;

        // ---- queries of rows r and r + 8, and what they see of the draft
        uint32_t qf[kQInSmem ? 1 : kSteps][4];
        uint64_t sees[2];
        const uint16_t* qp[2];
        bool live[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = r + 8 * i;
            live[i] = row < rows;
            const int node = live[i] ? (rt * kRows + row) / G : 0;
            const int head = live[i] ? hk * G + (rt * kRows + row) % G : 0;
            const int64_t t = seq.first + node;
            qp[i] = static_cast<const uint16_t*>(a.q) + t * a.ld_q + (int64_t)head * D;
            sees[i] = !live[i] ? 0 : a.mask ? (uint64_t)a.mask[t] : (2ull << node) - 1;
        }
        auto q_words = [&](int ks, uint32_t (&w)[4]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint2 x = make_uint2(0, 0);
                if (live[i]) x = *reinterpret_cast<const uint2*>(qp[i] + k_elem<E4M3>(ks, c));
                w[i] = E4M3 ? __byte_perm(x.x, x.y, 0x5410) : x.x;      // elements 0, 2 | 0, 1
                w[2 + i] = E4M3 ? __byte_perm(x.x, x.y, 0x7632) : x.y;  // elements 1, 3 | 2, 3
            }
        };
        if (kQInSmem) {
            for (int ks = warp; ks < kSteps; ks += kWarps) {
                uint32_t w[4];
                q_words(ks, w);
                *reinterpret_cast<uint4*>(q_smem + (ks * 32 + lane) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) q_words(ks, qf[ks]);
        }

        // ---- the ring: this warp's 16 tokens of tile `tile` into stage `st`
        const int64_t head_rows = (int64_t)hk << a.c.page_shift;
        auto issue = [&](int tile, int st) {
            const int pos = tile * kTile + warp * 16;
            uint8_t* dst = ring + st * C::kStage;
            if (tile < tile1) {
                // pages hold a multiple of 16 tokens: the whole step lies in one
                int64_t row = pos < seq.len ? page_row(a.p, a.c, seg.n, pos) : 0;
                const bool bad = row < 0;
                if (bad) {
                    if (lane == 0) set_status(a.status, kStatusBadSeqlens);
                    row = 0;
                }
                const int left = bad ? 0 : seq.len - pos;  // tokens of the step that exist
                row += bad || left <= 0 ? 0 : head_rows;
                const uint8_t* kb = static_cast<const uint8_t*>(a.c.k) + row * C::kRowBytes;
                const uint8_t* vb = static_cast<const uint8_t*>(a.c.v) + row * C::kRowBytes;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int tok = 8 * nt + r;
                    const bool on = tok < left;
#pragma unroll
                    for (int j = 0; j < C::kKChunks; ++j)
                        cp_async_zfill16(dst + ((nt * C::kKChunks + j) * 32 + lane) * 16,
                                         kb + (on ? tok : 0) * C::kRowBytes + 64 * j + 16 * c, on);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int tok = 2 * c + (x & 1) + 8 * (x >> 1);
                    const bool on = tok < left;
#pragma unroll
                    for (int j = 0; j < C::kVChunks; ++j) {
                        uint8_t* d = dst + C::kKStage + ((x * C::kVChunks + j) * 32 + lane) * C::kVBytes;
                        const uint8_t* s = vb + (on ? tok : 0) * C::kRowBytes + (8 * j + r) * C::kVBytes;
                        if (C::kVBytes == 16) cp_async_zfill16(d, s, on);
                        else cp_async_zfill8(d, s, on);
                    }
                }
                if (E4M3) {
                    const int tok = lane & 15;
                    const float* s = (lane < 16 ? a.c.k_scale : a.c.v_scale) + row + (tok < left ? tok : 0);
                    cp_async_zfill4(dst + C::kKStage + C::kVStage + 4 * lane, s, tok < left);
                }
            }
            cp_async_commit_group();
        };

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
        bool odd = false;  // a drafted value was not finite
        const float scale2 = a.scale * kLog2e;

#pragma unroll
        for (int st = 0; st < C::kStages - 1; ++st) issue(tile0 + st, st);
        int st = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            {
                int next = st + C::kStages - 1;
                if (next >= C::kStages) next -= C::kStages;
                __syncwarp();  // every lane has read the stage (its scales) that is filled next
                issue(tile + C::kStages - 1, next);
            }
            cp_async_wait_group<C::kStages - 1>();
            if (E4M3) __syncwarp();  // the scales were copied by other lanes
            const uint8_t* src = ring + st * C::kStage;
            if (++st == C::kStages) st = 0;
            const int pos = tile * kTile + warp * 16;
            if (pos >= seq.len) continue;

            // ---- scores: rows r, r + 8 x tokens 8 nt + 2c, + 1
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < C::kKChunks; ++j) {
                uint4 kw[2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
                    kw[nt] = *reinterpret_cast<const uint4*>(src + ((nt * C::kKChunks + j) * 32 + lane) * 16);
                constexpr int per = E4M3 ? 4 : 2;  // k-steps of a 16-byte piece
#pragma unroll
                for (int x = 0; x < per; ++x) {
                    uint32_t qa[4];
                    if (kQInSmem) {
                        const uint4 u = *reinterpret_cast<const uint4*>(q_smem + ((per * j + x) * 32 + lane) * 4);
                        qa[0] = u.x; qa[1] = u.y; qa[2] = u.z; qa[3] = u.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) qa[e] = qf[kQInSmem ? 0 : per * j + x][e];
                    }
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const uint32_t w[4] = {kw[nt].x, kw[nt].y, kw[nt].z, kw[nt].w};
                        uint32_t b0, b1;
                        if (E4M3) {
                            b0 = e4m3_hi_to_bf16x2(w[x] << 8);  // bytes 0, 2
                            b1 = e4m3_hi_to_bf16x2(w[x]);       // bytes 1, 3
                        } else {
                            b0 = w[2 * x];
                            b1 = w[2 * x + 1];
                        }
                        mma_16816(s[nt], qa, b0, b1);
                    }
                }
            }
            // ---- softmax in powers of two
            float vs[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                float2 k2 = make_float2(scale2, scale2);
                if (E4M3) {
                    const float* sc = reinterpret_cast<const float*>(src + C::kKStage + C::kVStage);
                    const float2 x = *reinterpret_cast<const float2*>(sc + 8 * nt + 2 * c);
                    const float2 y = *reinterpret_cast<const float2*>(sc + 16 + 8 * nt + 2 * c);
                    k2 = make_float2(x.x * scale2, x.y * scale2);
                    vs[nt][0] = y.x;
                    vs[nt][1] = y.y;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] *= e & 1 ? k2.y : k2.x;
            }
            const bool drafted = pos + 16 > base;  // some token is not every row's
            uint32_t on = 0xFFu;                   // bit nt * 4 + e
            if (drafted) {
                on = 0;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = pos + 8 * nt + 2 * c + (e & 1);
                        const bool see = t < base || (t < seq.len && ((sees[e >> 1] >> (t - base)) & 1));
                        if (see) on |= 1u << (nt * 4 + e);
                        else s[nt][e] = kNegInf;
                    }
            }
            float top[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                top[i] = fmaxf(m[i], x);
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f[i] = m[i] == kNegInf ? 0.f : exp2_approx(m[i] - top[i]);
                    l[i] *= f[i];
                    m[i] = top[i];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= f[0];
                    o[i][1] *= f[0];
                    o[i][2] *= f[1];
                    o[i][3] *= f[1];
                }
            }
            uint32_t pa[4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float ref = m[i] == kNegInf ? 0.f : m[i];
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[e] = exp2_approx(s[nt][2 * i + e] - ref);
                        l[i] += p[e];
                        // a token that the row does not see adds nothing, whatever its scale
                        if (E4M3) p[e] = (on >> (nt * 4 + 2 * i + e)) & 1 ? p[e] * vs[nt][e] : 0.f;
                    }
                    pa[2 * nt + i] = pack_bf16(p[0], p[1]);
                }
            // ---- outputs: tokens {2c, 2c + 1, 2c + 8, 2c + 9} x this lane's piece of d
#pragma unroll
            for (int j = 0; j < C::kVChunks; ++j) {
                constexpr int W = C::kVBytes / 4;
                uint32_t v[4][W];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint8_t* p = src + C::kKStage + ((x * C::kVChunks + j) * 32 + lane) * C::kVBytes;
                    if (W == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(p);
                        v[x][0] = u.x; v[x][1] = u.y; v[x][W > 2 ? 2 : 0] = u.z; v[x][W > 3 ? 3 : 1] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(p);
                        v[x][0] = u.x; v[x][1] = u.y;
                    }
                }
                if (!E4M3 && drafted) {
                    // a drafted value that is not finite must not reach the rows that do not see it:
                    // zero here, added to the others at the end of the segment
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            if ((v[x][w] & 0x7F80u) == 0x7F80u) v[x][w] &= 0xFFFF0000u, odd = true;
                            if ((v[x][w] & 0x7F800000u) == 0x7F800000u) v[x][w] &= 0x0000FFFFu, odd = true;
                        }
                }
                constexpr int per = E4M3 ? 4 : 2;  // elements of a word
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int e = 0; e < per; ++e) {
                        uint32_t b0, b1;
                        if (E4M3) {
                            const uint32_t sel = 0x4000u + (uint32_t)e * 0x1111u;  // byte 1: v0's, byte 3: v1's
                            b0 = e4m3_hi_to_bf16x2(__byte_perm(v[0][w], v[1][w], sel));
                            b1 = e4m3_hi_to_bf16x2(__byte_perm(v[2][w], v[3][w], sel));
                        } else {
                            b0 = __byte_perm(v[0][w], v[1][w], e ? 0x7632 : 0x5410);
                            b1 = __byte_perm(v[2][w], v[3][w], e ? 0x7632 : 0x5410);
                        }
                        mma_16816(o[j * C::kVElems + w * per + e], pa, b0, b1);
                    }
            }
        }
        cp_async_wait_group<0>();

        // ---- join the four warps: m, l and o of every row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        const bool any_odd = __syncthreads_or(odd);  // and the rings are drained: they hold the sums now
        float* buf = reinterpret_cast<float*>(smem);                  // [warp][row][D]
        float* mw = buf + kWarps * kRows * D;                         // [warp][row]
        float* lw = mw + kWarps * kRows;
        if (c == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mw[warp * kRows + r + 8 * i] = m[i];
                lw[warp * kRows + r + 8 * i] = l[i];
            }
        }
        __syncthreads();
        float top[2], f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = kNegInf;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top[i] = fmaxf(top[i], mw[w * kRows + r + 8 * i]);
            f[i] = m[i] == kNegInf ? 0.f : exp2_approx(m[i] - top[i]);
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            // column 2c + e of tile j: lane r = 2c + e of the value fragments, element j of its pieces
            const int piece = j / C::kVElems, x = j % C::kVElems;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (8 * piece + 2 * c + (e & 1)) * C::kVElems + x;
                buf[(warp * kRows + r + 8 * (e >> 1)) * D + d] = o[j][e] * f[e >> 1];
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == seg.tiles;
        float* part = partials + (2 * (int)blockIdx.x + seg.later) * slot_floats(D, a.slot_rows);
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), d = 4 * (x % (D / 4));
            float mt = kNegInf, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, mw[w * kRows + row]);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw_ = mw[w * kRows + row];
                lt += mw_ == kNegInf ? lw[w * kRows + row] : lw[w * kRows + row] * exp2_approx(mw_ - mt);
                const float4 z = *reinterpret_cast<const float4*>(buf + (w * kRows + row) * D + d);
                y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
            }
            const int node = (rt * kRows + row) / G, head = hk * G + (rt * kRows + row) % G;
            const int64_t t = seq.first + node;
            if (!E4M3 && any_odd) {
                // drafted values that are not finite, for the rows that see them
                const uint64_t bits = a.mask ? (uint64_t)a.mask[t] : (2ull << node) - 1;
                const int from = max(base, tile0 * kTile), to = min(seq.len, tile1 * kTile);
                for (int p = from; p < to; ++p) {
                    if (!((bits >> (p - base)) & 1)) continue;
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
            if (a.gate) {
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

// Joins the partials of the units that span CTAs: one warp per row.
template <int D, int ROWS, int TN>
__global__ void __launch_bounds__(kThreads) join_kernel(TreeArgs a) {
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x / a.c.Hk, hk = blockIdx.x % a.c.Hk;
    const int G = a.H / a.c.Hk;
    const int x = blockIdx.y * kWarps + (threadIdx.x >> 5);  // row of the (sequence, head)
    pdl_wait_previous();
    const Seq seq = load_seq(a, n);
    if (x >= seq.nodes * G) return;
    const int rt = x / ROWS, row = x % ROWS;
    const LineMeta line = line_meta(a)[rt];
    const int64_t tiles = seq_tiles<TN>(seq);
    const int64_t start = line_starts(a, rt)[n] + hk * tiles;
    const int64_t c0 = share_of(start, line.total, line.shares);
    const int64_t c1 = share_of(start + tiles - 1, line.total, line.shares);
    if (c0 == c1) return;  // one CTA had the whole unit and wrote it
    const float* partials = partial_base(a);
    auto part = [&](int64_t c) {
        const bool later = c == c0 && share_start(c0, line.total, line.shares) != start;
        return partials + (2 * (line.first_cta + c) + later) * slot_floats(D, a.slot_rows);
    };
    float mt = kNegInf, lt = 0.f;
    for (int64_t b = c0; b <= c1; b += 32) mt = fmaxf(mt, b + lane <= c1 ? part(b + lane)[row] : kNegInf);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    constexpr int V = D / 128 > 0 ? D / 128 : 1;  // float4s of a lane
    float4 y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t b = c0; b <= c1; b += 32) {
        float f = 0.f;
        if (b + lane <= c1) {
            const float* p = part(b + lane);
            const float mi = p[row];
            f = mi == kNegInf ? 1.f : exp2_approx(mi - mt);  // a part that saw nothing holds zeros (or NaN)
            lt += p[a.slot_rows + row] * f;
        }
        const int count = (int)(c1 - b + 1 < 32 ? c1 - b + 1 : 32);
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            const float* p = part(b + i) + 2 * a.slot_rows + row * D;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (4 * lane + 128 * v >= D) continue;
                const float4 z = *reinterpret_cast<const float4*>(p + 4 * lane + 128 * v);
                y[v].x = fmaf(z.x, fi, y[v].x); y[v].y = fmaf(z.y, fi, y[v].y);
                y[v].z = fmaf(z.z, fi, y[v].z); y[v].w = fmaf(z.w, fi, y[v].w);
            }
        }
    }
    lt = warp_sum(lt);
    const bool empty = mt == kNegInf && lt == 0.f;
    const float inv = empty ? 0.f : 1.f / lt;
    const int64_t t = seq.first + x / G;
    const int head = hk * G + x % G;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int d = 4 * lane + 128 * v;
        if (d >= D) continue;
        const int64_t out = (t * a.H + head) * D + d;
        float4 z = make_float4(y[v].x * inv, y[v].y * inv, y[v].z * inv, y[v].w * inv);
        if (a.gate) {
            const float4 g = load4(static_cast<const uint16_t*>(a.gate) + out);
            z.x /= 1.f + __expf(-g.x); z.y /= 1.f + __expf(-g.y);
            z.z /= 1.f + __expf(-g.z); z.w /= 1.f + __expf(-g.w);
        }
        store4(static_cast<uint16_t*>(a.o) + out, z);
    }
    if (a.lse && lane == 0) a.lse[t * a.H + head] = empty ? kNegInf : mt * kLn2 + logf(lt);
}

int sm_count() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int D>
int ctas_dim(int e4m3) {
    return e4m3 ? Config<D, true>::kCtas : Config<D, false>::kCtas;
}

// The launch's shape from its sizes alone.
struct Plan {
    bool tc;  // the tcgen05 kernel
    int grid, row_tiles, slot_rows, min_tiles;
};
Plan make_plan(int H, int Hk, int D, int max_nodes, int e4m3) {
    Plan p;
    const int rows = max_nodes * (H / Hk);
    p.tc = rows > kRows;
    const int tile = p.tc ? kTcRows : kRows;
    p.row_tiles = (rows + tile - 1) / tile;
    p.slot_rows = ((rows < tile ? rows : tile) + 3) / 4 * 4;
    p.grid = sm_count() * (p.tc ? 1 : D == 64 ? ctas_dim<64>(e4m3) : D == 128 ? ctas_dim<128>(e4m3) : ctas_dim<256>(e4m3));
    if (p.grid < p.row_tiles) p.grid = p.row_tiles;
    p.min_tiles = p.tc ? 1 : 2;
    return p;
}

template <int D, bool E4M3>
cudaError_t launch_config(const TreeArgs& a, bool tc, cudaStream_t s) {
    using C = Config<D, E4M3>;
    cudaError_t e;
    const int rows = a.max_nodes * (a.H / a.c.Hk);
    const dim3 join(a.p.N * a.c.Hk, (rows + kWarps - 1) / kWarps);
    if (tc) {
        if ((e = launch_tree_tc(a, s)) != cudaSuccess) return e;
        return launch_pdl(join_kernel<D, kTcRows, (D == 256 ? 64 : 128)>, join, dim3(kThreads), 0, s, a);
    }
    e = cudaFuncSetAttribute(tree_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    tree_kernel<D, E4M3><<<a.grid, kThreads, C::kSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_pdl(join_kernel<D, kRows, kTile>, join, dim3(kThreads), 0, s, a);
}

template <int D>
cudaError_t launch_dim(const TreeArgs& a, bool tc, cudaStream_t s) {
    return a.c.e4m3 ? launch_config<D, true>(a, tc, s) : launch_config<D, false>(a, tc, s);
}

}  // namespace

size_t tree_workspace_bytes(int N, int H, int Hk, int D, int max_nodes, int e4m3) {
    const Plan p = make_plan(H, Hk, D, max_nodes, e4m3);
    return meta_bytes(p.row_tiles, N) + 2 * (size_t)p.grid * slot_floats(D, p.slot_rows) * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeArgs& args, cudaStream_t s) {
    TreeArgs a = args;
    const Plan p = make_plan(a.H, a.c.Hk, a.c.D, a.max_nodes, a.c.e4m3);
    a.grid = p.grid;
    a.row_tiles = p.row_tiles;
    a.slot_rows = p.slot_rows;
    a.min_tiles = p.min_tiles;
    return a.c.D == 64 ? launch_dim<64>(a, p.tc, s) : a.c.D == 128 ? launch_dim<128>(a, p.tc, s) : launch_dim<256>(a, p.tc, s);
}

}  // namespace gdn
