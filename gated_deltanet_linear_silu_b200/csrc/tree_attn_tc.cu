// Attention of a drafted tree over the paged cache, on the tensor cores' tcgen05
// path (formula in tree_attn.cu).
//
// A unit is (sequence, key/value head, 128 query rows): rows are (node, query
// head of the group) pairs, the M side of the products. One persistent CTA per
// SM walks an equal share of the 128-token (D = 256: 64-token) tiles of its row
// tile's line; 13 warps:
//   warps 0-3   softmax, a row per thread: scores from tensor memory, running
//               maximum and sum, probabilities back to tensor memory as bf16;
//               the output at the end of a segment
//   warp 4      issues the products: S = Q K^T of tile i + 1 goes out before
//               O += P V of tile i, so that the next scores form meanwhile
//   warps 5-12  producers: cache rows (page by page) into the shared-memory
//               tiles the products read. bf16 rows by cp.async; e4m3 rows
//               through registers (the loads of the next tile in flight while
//               this one is converted), bf16 exactly
// The output accumulates in tensor memory under a reference maximum that is
// only moved (and the output rescaled) when a row's maximum outgrows it by 2^8,
// which fp32 sums and bf16's exponent range absorb.
//
// Every wait is bounded (gdn_set_wait_limit_ns).
#include <cfloat>

#include "kv_page.cuh"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kSoftWarps = 4, kMmaWarp = 4, kProdWarp0 = 5, kProdWarps = 8;
constexpr int kTcThreads = 32 * (kProdWarp0 + kProdWarps);
constexpr int kProdThreads = 32 * kProdWarps;
constexpr int kScaleSlots = 4;
constexpr uint64_t kDrainWaitNs = 1000000000ull;

template <int D>
struct Tc {
    static constexpr int TN = D == 256 ? 64 : 128;  // tokens of a tile
    static constexpr int kBlockQ = kTcRows * 128;   // 64 elements of every row
    static constexpr int kBlock = TN * 128;
    static constexpr int kBlocks = D / 64;
    static constexpr int kQ = kBlockQ * kBlocks, kTileBytes = kBlock * kBlocks;
    static constexpr int kOffK = kQ, kOffV = kOffK + 2 * kTileBytes, kOffScale = kOffV + 2 * kTileBytes;
    static constexpr int kOffBars = kOffScale + kScaleSlots * 2 * TN * 4;
    static constexpr int kUsed = kOffBars + 256 + 1024;  // 1024: alignment
    // above half of the SM's shared memory, so that a CTA has its tensor memory to itself
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static constexpr int kColS = D == 256 ? 256 : 128;  // S buffers behind O
    static constexpr uint32_t kIdescS = idesc_bf16(128, TN, 0, 0);
    static constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1);
};

struct TcBars {
    uint64_t kfull[2], kempty[2];  // producers (8 warps) / commit
    uint64_t vfull[2], vempty[2];
    uint64_t sfull[2];             // scores of a tile (commit)
    uint64_t pfull[2];             // its probabilities (4 warps)
    uint64_t odone;                // output product of a tile done (commit)
    uint64_t ofree;                // a segment's output read (4 warps)
    uint64_t qfull, qempty;        // a segment's queries (8 warps / commit)
    uint64_t cfull[kScaleSlots];   // a tile's scales (8 warps)
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int odd;                       // some drafted value was not finite
};
static_assert(sizeof(TcBars) <= 256, "barrier block");

__device__ __noinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    if (limit == 0) return mbar_test_wait(bar, parity);
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        for (int k = 0; k < 32; ++k)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag || globaltimer_ns() - t0 > limit) return false;
    }
}

// The same for a whole warp: one lane waits, all of them learn the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    const bool ok = (threadIdx.x & 31) != 0 || tc_wait(bar, parity, abort_flag, limit);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// The bits of 32 positions from offset `off` past the context: what a row sees.
__device__ __forceinline__ uint32_t sees32(uint64_t sees, int off) {
    if (off <= -32) return 0xFFFFFFFFu;
    if (off >= 64) return 0u;
    if (off >= 0) return (uint32_t)(sees >> off);
    return (uint32_t)(sees << -off) | ((1u << -off) - 1u);
}

// 16 e4m3 codes as 16 bf16, each four in the order 0, 2, 1, 3.
__device__ __forceinline__ void convert16(const uint4& u, uint4 (&out)[2]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = e4m3_hi_to_bf16x2(w[i] << 8);
        y[2 * i + 1] = e4m3_hi_to_bf16x2(w[i]);
    }
    out[0] = make_uint4(y[0], y[1], y[2], y[3]);
    out[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTcThreads, 1) tree_tc_kernel(TreeArgs a) {
    using C = Tc<D>;
    constexpr int TN = C::TN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TcBars& B = *reinterpret_cast<TcBars*>(sm + C::kOffBars);
    volatile int* abort_flag = &B.abort_flag;
    float* scales = reinterpret_cast<float*>(sm + C::kOffScale);  // [slot][k then v][TN]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.H / a.c.Hk;
    const uint64_t wlim = a.wait_ns;
    pdl_launch_dependents();

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.kfull[i], kProdWarps);
            mbar_init(&B.kempty[i], 1);
            mbar_init(&B.vfull[i], kProdWarps);
            mbar_init(&B.vempty[i], 1);
            mbar_init(&B.sfull[i], 1);
            mbar_init(&B.pfull[i], kSoftWarps);
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&B.cfull[i], kProdWarps);
        mbar_init(&B.odone, 1);
        mbar_init(&B.ofree, kSoftWarps);
        mbar_init(&B.qfull, kProdWarps);
        mbar_init(&B.qempty, 1);
        mbar_init(&B.drain, 1);
        fence_mbar_init();
        B.abort_flag = 0;
        B.odd = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&B.tmem, 512);
    tc_fence_before();
    const Share share = find_share<kTcRows, TN, kTcThreads>(a);
    tc_fence_after();  // (find_share synchronises the CTA)
    const uint32_t tmem = B.tmem;
    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            set_status(a.status, kStatusTimeout);
        }
    };

    if (warp >= kProdWarp0) {
        // ============================================================ producers
        const int pt = tid - 32 * kProdWarp0;
        constexpr int kElem = E4M3 ? 1 : 2;
        constexpr int kPer = D * kElem / 16;                     // 16-byte pieces of a row
        constexpr int kPieces = TN * kPer / kProdThreads;        // of a thread, per tile
        constexpr int kTokStep = kProdThreads / kPer;            // tokens between its pieces
        const int tok0 = pt / kPer, col = pt % kPer;
        bool ok = true;
        int64_t i = 0;  // tile number in this CTA
        int seg_no = 0;
        Segment seg;
        bool have = first_segment<kTcRows, TN>(a, share, seg);
        // Cache row of each of this thread's tokens of the tile at pos, -1: zeros.
        // (The C ABI keeps a cache's rows below 2^31.)
        auto rows_of = [&](const Segment& g, int pos, int (&row)[kPieces]) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int p = pos + tok0 + j * kTokStep;
                row[j] = -1;
                if (p < g.seq.len) {
                    row[j] = (int)page_row(a.p, a.c, g.n, p);
                    if (row[j] < 0) set_status(a.status, kStatusBadSeqlens);
                    else row[j] += g.hk << a.c.page_shift;
                }
            }
        };
        auto load_queries = [&](const Segment& g) -> bool {
            if (seg_no > 0 && !warp_wait(&B.qempty, (seg_no - 1) & 1, abort_flag, wlim)) return false;
            for (int x = pt; x < kTcRows * (D / 8); x += kProdThreads) {
                const int m = x / (D / 8), c8 = x % (D / 8);
                uint4 u = make_uint4(0, 0, 0, 0);
                if (m < g.rows) {
                    const int r = g.rt * kTcRows + m;
                    const int64_t t = g.seq.first + r / G;
                    u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + t * a.ld_q +
                                                       (int64_t)(g.hk * G + r % G) * D + 8 * c8);
                    if (E4M3)
                        u = make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632),
                                       __byte_perm(u.z, u.w, 0x5410), __byte_perm(u.z, u.w, 0x7632));
                }
                *reinterpret_cast<uint4*>(sm + (c8 >> 3) * C::kBlockQ + sw128_off(m, c8 & 7)) = u;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.qfull);
            return true;
        };
        auto publish = [&](uint64_t* bar) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        if (E4M3) {
            uint4 kr[kPieces], vr[kPieces];
            float ks = 0.f, vs = 0.f;
            int row[kPieces];
            const float scale2 = a.scale * kLog2e;
            auto load_k = [&]() {
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    kr[j] = row[j] < 0 ? make_uint4(0, 0, 0, 0)
                                       : __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.k) + (int64_t)row[j] * D) + col);
            };
            auto load_v = [&]() {
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    vr[j] = row[j] < 0 ? make_uint4(0, 0, 0, 0)
                                       : __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.v) + (int64_t)row[j] * D) + col);
            };
            auto load_scales = [&](const Segment& g, int pos) {
                if (pt < TN) {
                    ks = vs = 0.f;
                    if (pos + pt < g.seq.len) {
                        int64_t r = page_row(a.p, a.c, g.n, pos + pt);
                        if (r >= 0) {
                            r += (int64_t)g.hk << a.c.page_shift;
                            ks = __ldg(a.c.k_scale + r) * scale2;
                            vs = __ldg(a.c.v_scale + r);
                        }
                    }
                }
            };
            auto store = [&](uint8_t* tile, const uint4 (&x)[kPieces]) {
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    uint4 y[2];
                    convert16(x[j], y);
                    const int tok = tok0 + j * kTokStep;
                    uint8_t* p = tile + (col >> 2) * C::kBlock;
                    // neighbouring blocks start with the other half: eight lanes, eight banks groups
                    const int f = (col >> 2) & 1, c16 = 2 * (col & 3);
                    *reinterpret_cast<uint4*>(p + sw128_off(tok, c16 + f)) = f ? y[1] : y[0];
                    *reinterpret_cast<uint4*>(p + sw128_off(tok, c16 + 1 - f)) = f ? y[0] : y[1];
                }
            };
            int tile = 0;
            if (have) {
                tile = seg.tile0;
                rows_of(seg, tile * TN, row);
                load_scales(seg, tile * TN);
                load_k();
                load_v();
            }
            while (ok && have) {
                if (tile == seg.tile0 && !load_queries(seg)) { ok = false; break; }
                const int st = (int)(i & 1), par = (int)((i >> 1) & 1);
                // the tile after this one
                Segment next = seg;
                int next_tile = tile + 1;
                bool more = true;
                if (next_tile == seg.tile1) {
                    more = next_segment<kTcRows, TN>(a, share, next);
                    next_tile = next.tile0;
                }
                if (!warp_wait(&B.kempty[st], par ^ 1, abort_flag, wlim)) { ok = false; break; }
                store(sm + C::kOffK + st * C::kTileBytes, kr);
                if (pt < TN) {
                    float* s = scales + (i % kScaleSlots) * 2 * TN;
                    s[pt] = ks;
                    s[TN + pt] = vs;
                }
                publish(&B.kfull[st]);
                if (lane == 0) mbar_arrive(&B.cfull[i % kScaleSlots]);
                if (more) {
                    rows_of(next, next_tile * TN, row);
                    load_scales(next, next_tile * TN);
                    load_k();
                }
                if (!warp_wait(&B.vempty[st], par ^ 1, abort_flag, wlim)) { ok = false; break; }
                store(sm + C::kOffV + st * C::kTileBytes, vr);
                publish(&B.vfull[st]);
                if (more) load_v();
                ++i;
                if (next_tile == next.tile0 && more) ++seg_no;
                seg = next;
                tile = next_tile;
                have = more;
            }
        } else {
            // groups of copies in order K0, V0, K1, V1, ...: a group is published once the two
            // issued after it are under way
            int64_t issued = 0, done = 0;  // groups; K and V of the CTA's tile x are 2 x and 2 x + 1
            int drafts[2] = {0, 0};        // of a V stage: 0, or its first drafted token's place + 1
            auto copy = [&](uint8_t* tile, const void* src, const int (&row)[kPieces]) {
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const uint8_t* s = static_cast<const uint8_t*>(src) + (int64_t)(row[j] < 0 ? 0 : row[j]) * (2 * D) + 16 * col;
                    cp_async_zfill16(tile + (col >> 3) * C::kBlock + sw128_off(tok0 + j * kTokStep, col & 7), s,
                                     row[j] >= 0);
                }
                cp_async_commit_group();
            };
            // Publishes group g; drafted values that are not finite become zero first (the rows that
            // see them get them at the end of the segment).
            auto finish = [&](int64_t g) {
                const int st = (int)((g >> 1) & 1);
                if (g & 1) {
                    const int draft_pos = drafts[st];
                    if (draft_pos) {
                        uint8_t* tile = sm + C::kOffV + st * C::kTileBytes;
                        bool odd = false;
#pragma unroll
                        for (int j = 0; j < kPieces; ++j) {
                            const int tok = tok0 + j * kTokStep;
                            if (tok < draft_pos - 1) continue;
                            uint32_t* w = reinterpret_cast<uint32_t*>(tile + (col >> 3) * C::kBlock + sw128_off(tok, col & 7));
                            for (int e = 0; e < 4; ++e) {
                                uint32_t x = w[e];
                                const uint32_t y = x;
                                if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
                                if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
                                if (x != y) {
                                    w[e] = x;
                                    odd = true;
                                }
                            }
                        }
                        if (odd) *reinterpret_cast<volatile int*>(&B.odd) = 1;
                    }
                    publish(&B.vfull[st]);
                } else {
                    publish(&B.kfull[st]);
                }
            };
            while (ok && have) {
                if (!load_queries(seg)) { ok = false; break; }
                const int base = seg.seq.len - seg.seq.nodes;
                for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++i) {
                    const int st = (int)(i & 1), par = (int)((i >> 1) & 1);
                    int row[kPieces];
                    rows_of(seg, tile * TN, row);
                    if (!warp_wait(&B.kempty[st], par ^ 1, abort_flag, wlim)) { ok = false; break; }
                    copy(sm + C::kOffK + st * C::kTileBytes, a.c.k, row);
                    if (++issued - done > 2) {
                        cp_async_wait_group<2>();
                        finish(done++);
                    }
                    if (!warp_wait(&B.vempty[st], par ^ 1, abort_flag, wlim)) { ok = false; break; }
                    const int from = base - tile * TN;  // the draft's first token in this tile
                    drafts[st] = from < TN ? (from > 0 ? from : 0) + 1 : 0;
                    copy(sm + C::kOffV + st * C::kTileBytes, a.c.v, row);
                    if (++issued - done > 2) {
                        cp_async_wait_group<2>();
                        finish(done++);
                    }
                }
                if (!ok) break;
                // nothing may hold back the segment's last groups: the next one's queries wait for them
                cp_async_wait_group<0>();
                while (done < issued) finish(done++);
                ++seg_no;
                have = next_segment<kTcRows, TN>(a, share, seg);
            }
        }
        if (!ok) fail();
        cp_async_wait_group<0>();
    } else if (warp == kMmaWarp) {
        // ================================================================ products
        if (lane == 0) {
            bool ok = true;
            Segment seg;
            bool have = first_segment<kTcRows, TN>(a, share, seg);
            int64_t i = 0;
            int seg_no = 0;
            auto scores = [&](int64_t x, bool first, bool last, int sn) -> bool {  // S of tile x
                const int st = (int)(x & 1);
                if (first && !tc_wait(&B.qfull, sn & 1, abort_flag, wlim)) return false;
                if (!tc_wait(&B.kfull[st], (x >> 1) & 1, abort_flag, wlim)) return false;
                tc_fence_after();
                const uint32_t k0 = smem_u32(sm + C::kOffK + st * C::kTileBytes), q0 = smem_u32(sm);
#pragma unroll 4
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16(tmem + C::kColS + st * TN, sw128_desc(q0 + (kk >> 2) * C::kBlockQ + 32 * (kk & 3), 16, 1024),
                             sw128_desc(k0 + (kk >> 2) * C::kBlock + 32 * (kk & 3), 16, 1024), C::kIdescS, kk > 0);
                mma_commit(&B.sfull[st]);
                mma_commit(&B.kempty[st]);
                if (last) mma_commit(&B.qempty);
                return true;
            };
            if (have) ok = scores(0, true, seg.tile1 - seg.tile0 == 1, 0);
            int tile = have ? seg.tile0 : 0;
            while (ok && have) {
                Segment next = seg;
                int next_tile = tile + 1;
                const bool crosses = next_tile == seg.tile1;
                bool more = true;
                if (crosses) {
                    more = next_segment<kTcRows, TN>(a, share, next);
                    next_tile = next.tile0;
                }
                if (!crosses && !scores(i + 1, false, next_tile + 1 == seg.tile1, seg_no)) { ok = false; break; }
                const int st = (int)(i & 1);
                if (tile == seg.tile0 && seg_no > 0 && !tc_wait(&B.ofree, (seg_no - 1) & 1, abort_flag, wlim)) {
                    ok = false;
                    break;
                }
                if (!tc_wait(&B.pfull[st], (i >> 1) & 1, abort_flag, wlim) ||
                    !tc_wait(&B.vfull[st], (i >> 1) & 1, abort_flag, wlim)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t v0 = smem_u32(sm + C::kOffV + st * C::kTileBytes);
#pragma unroll 4
                for (int kk = 0; kk < TN / 16; ++kk)
                    mma_bf16_ta(tmem, tmem + C::kColS + st * TN + 8 * kk, sw128_desc(v0 + 2048 * kk, C::kBlock, 1024),
                                C::kIdescO, tile != seg.tile0 || kk > 0);
                mma_commit(&B.odone);
                mma_commit(&B.vempty[st]);
                if (crosses && more) {
                    ++seg_no;
                    if (!scores(i + 1, true, next.tile1 - next.tile0 == 1, seg_no)) { ok = false; break; }
                }
                ++i;
                seg = next;
                tile = next_tile;
                have = more;
            }
            if (!ok) fail();
            mma_commit(&B.drain);
            mbar_wait(&B.drain, 0, kDrainWaitNs);
        }
        __syncwarp();
    } else {
        // ================================================================= softmax
        const int m = tid;  // row of the tile, lane of tensor memory
        const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
        bool ok = true;
        int64_t i = 0;
        Segment seg;
        for (bool have = first_segment<kTcRows, TN>(a, share, seg); ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
            const bool busy = 32 * warp < seg.rows, live = m < seg.rows;
            const int r = seg.rt * kTcRows + (live ? m : 0);
            const int node = r / G, head = seg.hk * G + r % G;
            const int64_t t = seg.seq.first + node;
            const int base = seg.seq.len - seg.seq.nodes;
            uint64_t sees = 0;
            if (live) {
                sees = a.mask ? (uint64_t)a.mask[t] : (2ull << node) - 1;
                if (seg.seq.nodes < 64) sees &= (1ull << seg.seq.nodes) - 1;
            }
            float ref = kNegInf, l = 0.f;  // reference maximum (log2 units), sum
            const float scale2 = a.scale * kLog2e;
            for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++i) {
                const int st = (int)(i & 1);
                if (!warp_wait(&B.sfull[st], (i >> 1) & 1, abort_flag, wlim) ||
                    (E4M3 && !warp_wait(&B.cfull[i % kScaleSlots], (i / kScaleSlots) & 1, abort_flag, wlim))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (busy) {
                    const uint32_t s0 = tmem + lane_off + C::kColS + st * TN;
                    const float* sc = scales + (i % kScaleSlots) * 2 * TN;
                    const int off = tile * TN - base;  // the tile's start past the context
                    const bool masked = off + TN > 0;
                    float top = kNegInf;
#pragma unroll
                    for (int c0 = 0; c0 < TN; c0 += 32) {
                        float s[32];
                        tmem_ld32(s0 + c0, s);
                        tmem_wait_ld();
                        if (E4M3) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 k4 = *reinterpret_cast<const float4*>(sc + c0 + e);
                                s[e] *= k4.x; s[e + 1] *= k4.y; s[e + 2] *= k4.z; s[e + 3] *= k4.w;
                            }
                        }
                        if (masked) {
                            const uint32_t bits = sees32(sees, off + c0);
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[e] = (bits >> e) & 1 ? s[e] : kNegInf;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) top = max3(top, s[e], s[e + 1]);
                    }
                    if (!E4M3) top *= scale2;
                    // ---- the reference: moved when outgrown
                    const bool move = ref == kNegInf ? top > kNegInf : top > ref + kLazy;
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = move && ref != kNegInf ? exp2_approx(ref - top) : 1.f;
                        if (move) ref = top;
                        l *= f;
                        if (tile != seg.tile0 && __any_sync(0xffffffffu, f != 1.f)) {
                            if (!warp_wait(&B.odone, (i - 1) & 1, abort_flag, wlim)) { ok = false; break; }
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 32) {
                                float o[32];
                                tmem_ld32(tmem + lane_off + c0, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= f;
                                tmem_st32(tmem + lane_off + c0, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float minus = ref == kNegInf ? 0.f : -ref;
#pragma unroll
                    for (int c0 = 0; c0 < TN; c0 += 32) {
                        float s[32];
                        tmem_ld32(s0 + c0, s);
                        tmem_wait_ld();
                        const uint32_t bits = masked ? sees32(sees, off + c0) : 0xFFFFFFFFu;
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float4 k4 = make_float4(scale2, scale2, scale2, scale2), v4 = make_float4(1.f, 1.f, 1.f, 1.f);
                            if (E4M3) {
                                k4 = *reinterpret_cast<const float4*>(sc + c0 + e);
                                v4 = *reinterpret_cast<const float4*>(sc + TN + c0 + e);
                            }
                            const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, vv[4] = {v4.x, v4.y, v4.z, v4.w};
                            float w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                float q = exp2_approx(fmaf(s[e + x], kk[x], minus));
                                if (masked && !((bits >> (e + x)) & 1)) q = 0.f;
                                l += q;
                                w[x] = E4M3 ? q * vv[x] : q;
                                if (E4M3 && masked && !((bits >> (e + x)) & 1)) w[x] = 0.f;
                            }
                            p[e / 2] = pack_bf16(w[0], w[1]);
                            p[e / 2 + 1] = pack_bf16(w[2], w[3]);
                        }
                        tmem_st16(s0 + c0 / 2, p);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.pfull[st]);
            }
            if (!ok) break;
            // ---- the segment's output
            if (!warp_wait(&B.odone, (i - 1) & 1, abort_flag, wlim)) { ok = false; break; }
            tc_fence_after();
            const bool odd = !E4M3 && *reinterpret_cast<volatile int*>(&B.odd) != 0;
            if (busy) {
                const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
                const bool empty = ref == kNegInf && l == 0.f;
                const float inv = empty ? 0.f : 1.f / l;
                const int64_t out = (t * a.H + head) * D;
                float* part = partial_base(a) + (2 * (int64_t)blockIdx.x + seg.later) * slot_floats(D, a.slot_rows);
                if (!whole && live) {
                    part[m] = ref;
                    part[a.slot_rows + m] = l;
                }
                part += 2 * a.slot_rows + m * D;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float o[32];
                    tmem_ld32(tmem + lane_off + c0, o);
                    tmem_wait_ld();
                    if (E4M3) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {  // back to the elements' order
                            const float x = o[e + 1];
                            o[e + 1] = o[e + 2];
                            o[e + 2] = x;
                        }
                    }
                    if (!live) continue;
                    if (odd) {
                        const int from = max(base, seg.tile0 * TN), to = min(seg.seq.len, seg.tile1 * TN);
                        for (int p = from; p < to; ++p) {
                            if (!((sees >> (p - base)) & 1)) continue;
                            const int64_t vr = page_row(a.p, a.c, seg.n, p);
                            if (vr < 0) continue;
                            const uint16_t* v = static_cast<const uint16_t*>(a.c.v) +
                                                (vr + ((int64_t)seg.hk << a.c.page_shift)) * D + c0;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = bf16_to_f32(v[e]);
                                if (!(fabsf(x) <= FLT_MAX)) o[e] += x;
                            }
                        }
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(part + c0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= inv;
                    if (a.gate) {
                        const uint16_t* g = static_cast<const uint16_t*>(a.gate) + out + c0;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 z = load4(g + e);
                            o[e] /= 1.f + __expf(-z.x); o[e + 1] /= 1.f + __expf(-z.y);
                            o[e + 2] /= 1.f + __expf(-z.z); o[e + 3] /= 1.f + __expf(-z.w);
                        }
                    }
                    uint16_t* y = static_cast<uint16_t*>(a.o) + out + c0;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(y + e) = make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]),
                                                                     pack_bf16(o[e + 4], o[e + 5]), pack_bf16(o[e + 6], o[e + 7]));
                }
                if (whole && live && a.lse) a.lse[t * a.H + head] = empty ? kNegInf : ref * kLn2 + logf(l);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.ofree);
        }
        if (!ok) fail();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool E4M3>
cudaError_t launch_tc(const TreeArgs& a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D, E4M3><<<a.grid, kTcThreads, Tc<D>::kSmem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s) {
    switch (a.c.D) {
        case 64: return a.c.e4m3 ? launch_tc<64, true>(a, s) : launch_tc<64, false>(a, s);
        case 128: return a.c.e4m3 ? launch_tc<128, true>(a, s) : launch_tc<128, false>(a, s);
        default: return a.c.e4m3 ? launch_tc<256, true>(a, s) : launch_tc<256, false>(a, s);
    }
}

}  // namespace gdn
