// Attention of a drafted tree over the paged cache, on the tensor cores' tcgen05
// path (formula in tree_attn.cu): more than 16 query rows of a key/value head.
//
// A unit is (sequence, key/value head, 128 query rows), rows the M side of the
// products. One persistent CTA per SM walks an equal share of its row tile's
// line in tiles of TN tokens; 12 warps (bf16) or 16 (e4m3):
//   warps 0-7    softmax, a row per thread, four warps to a tile: even tiles and
//                odd tiles have their own running state and output accumulator
//                (D <= 128), so that one group's exponentials run beside the
//                other's maxima and neither waits for it. For D = 256 the two
//                accumulators do not fit: two warps share 32 rows and take half
//                of every tile each. Probabilities go back to tensor memory
//   warp 8       issues the products: S = Q K^T of tile i + 1 goes out before
//                O += P V of tile i
//   warp 9       loader: the tile's pages, a lane per page. bf16 tiles go
//                straight to their slots by TMA (128-byte swizzle); e4m3 pages
//                by bulk copies into a raw ring
//   from 10      converters. e4m3: raw tiles to f16 (exact) in the layout of the
//                products; bf16: the tiles that hold drafted tokens or end the
//                sequence, where rows past its end and drafted values that are
//                not finite must be zero
//   from 14      e4m3: the tile's scales, of keys and of values, and the latter's
//                logarithms
// Probabilities (and queries, where tensor memory has room) are the products' A
// operands in tensor memory: shared memory carries the copies, the conversion
// and the products' other operand, and is the next limit.
// Tiles stand in one ring of slots in the order K0, V0, K1, V1, ..., so that the
// keys of the next tiles do not wait for the values of this one.
//
// Scales, f16 and the reference R are those of tree_attn.cu. Where two warps
// share a row's reference (D = 256) they vote at a named barrier on whether it
// has to move, and only then exchange maxima and rescale the output.
//
// What bounds it. bf16, 8 sequences of 32768 tokens, 64 nodes, 4 x 8 heads of 128:
// 284 to 296 us (950 TFLOP/s, and 3.7 TB/s of a cache that is read once), 905 cycles a
// tile, all of them the issuing warp's: the products' 512 and three waits. The
// exponentials, 16 a cycle and SM, would take 512. The same from e4m3: 342 us, the
// converters'. Heads of 256 from e4m3 (24 ragged sequences up to 16389 tokens,
// 17 nodes): 81 to 90 us, 2190 cycles a tile, 1300 of them the converters' stores and
// 900 their waits and hand-overs (shared memory alone needs 1200), and 8 us of
// bounds, queries and output for each (sequence, head) that a CTA takes part in.
//
// Every wait between warps is bounded by gdn_set_wait_limit_ns, and the two at the
// end, for the copies and the products in flight, by kDrainWaitNs: nothing may land
// in the CTA's memory after it is gone. Either kind reports that it ran out.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <mutex>

#include "kv_page.cuh"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kConvWarp0 = 10;
constexpr int kScaleSlots = 8;  // tiles whose scales are kept
constexpr uint64_t kDrainWaitNs = 1000000000ull;

constexpr int TN = kTcTile;

template <int D, bool E4M3>
struct Tc {
    static constexpr bool kGroups = D <= 128;  // even and odd tiles apart
    // bf16 needs few converters, and 12 warps leave 168 registers to a thread;
    // 13 to 16 warps leave 128
    static constexpr int kConvWarps = E4M3 ? 4 : 2, kScaleWarps = E4M3 ? 2 : 0;
    static constexpr int kScaleWarp0 = kConvWarp0 + kConvWarps;
    static constexpr int kThreads = 32 * (kScaleWarp0 + kScaleWarps);
    static constexpr int kBlock = TN * 128;  // 64 elements of every row, 128-byte swizzled
    static constexpr int kBlocks = D / 64;
    static constexpr int kSlot = kBlock * kBlocks;
    static constexpr int kSlots = D == 256 ? (E4M3 ? 4 : 6) : (E4M3 ? 8 : 12);  // (even: two to a tile)
    // A tile's keys and values under one barrier: a wait and a hand-over fewer. Not
    // where only two tiles fit the ring and the values, converted last, would hold
    // up the scores.
    static constexpr bool kOneFull = !(E4M3 && D == 256);
    // raw e4m3 tiles: rows of D bytes of keys, then of values, then their scales
    static constexpr int kRaw = 2 * (TN * D + TN * 4), kRawSlots = E4M3 ? (D == 256 ? 2 : 3) : 1;
    static constexpr int kOffRaw = kSlots * kSlot;
    static constexpr int kOffScale = kOffRaw + (E4M3 ? kRawSlots * kRaw : 0);  // [slot][k, v, log2 v][TN]
    static constexpr int kScaleBytes = E4M3 ? kScaleSlots * 3 * TN * 4 : 0;
    static constexpr int kOffRows = kOffScale + kScaleBytes;  // what two warps tell each other: [2][2][128]
    static constexpr int kOffBars = kOffRows + 4 * 128 * 4;
    static constexpr int kUsed = kOffBars + 704 + 1024;       // 1024: alignment
    // above half of the SM's shared memory, so that a CTA has its tensor memory to itself
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem + 512 <= 227 * 1024, "shared memory");
    // A tile's scales are written as soon as its raw slot is full, which is when the
    // tile before it in that slot is converted, and that when the tile before it in
    // the products' slots is done: the scales of that one are read.
    static_assert(!E4M3 || kScaleSlots >= kRawSlots + kSlots / 2, "scales");
    // tensor memory: O (one or two), the queries, two or three buffers of S
    static constexpr int kBufs = kGroups ? 3 : 2;
    static constexpr int kColQ = kGroups ? 2 * D : D, kColS = kColQ + D / 2;
    static_assert(kColS + kBufs * TN <= 512, "tensor memory");
    static constexpr uint32_t kFormat = E4M3 ? ~((1u << 7) | (1u << 10)) : ~0u;  // f16 operands: format bits 0
    static constexpr uint32_t kIdescS = idesc_bf16(128, TN, 0, 0) & kFormat;
    static constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1) & kFormat;
};

struct TcBars {
    uint64_t full[12], empty[12];    // slots of the products (converter warps, bf16: or as many by the loader / commit)
    uint64_t hand[12];               // bf16: tile left to the converters (loader)
    uint64_t rfull[3], rempty[3];    // raw slots (bulk copies / converter and scale warps)
    uint64_t cfull[kScaleSlots];     // a tile's scales (scale warps)
    uint64_t sfull[3], pfull[3];     // scores (commit), probabilities (4 or 8 warps)
    uint64_t odone[2];               // output product of a tile done, per accumulator (commit)
    uint64_t oend, ofree;            // of a segment: all of them done (commit), output read (8 warps)
    uint64_t qfull;                  // queries in tensor memory (8 warps)
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int odd;                         // some drafted value was not finite
    int gave_up[kSoftWarps];         // a softmax warp whose wait ran out, for its partner
};
static_assert(sizeof(TcBars) <= 704, "barrier block");

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
// All lanes of a warp wait alike; the first probe is inline.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag, limit));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t y;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(y));
    return y != 0;
}
// The 64 softmax threads of two warps with the same rows, at their named barrier.
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return y != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&y);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&y);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(y)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&y);
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

template <int D, bool E4M3>
__global__ void __launch_bounds__((Tc<D, E4M3>::kThreads), 1)
tree_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v) {
    using C = Tc<D, E4M3>;
    constexpr int kConvWarps = C::kConvWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TcBars& B = *reinterpret_cast<TcBars*>(sm + C::kOffBars);
    volatile int* abort_flag = &B.abort_flag;
    float* scales = reinterpret_cast<float*>(sm + C::kOffScale);
    float* row_top = reinterpret_cast<float*>(sm + C::kOffRows);  // [half or group][row]
    float* row_sum = row_top + 256;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (warp-uniform to the compiler)
    const int G = a.H / a.c.Hk;
    const uint64_t wlim = a.wait_ns;
    if (tid == 0) {
        for (int i = 0; i < 12; ++i) {
            mbar_init(&B.full[i], kConvWarps);
            mbar_init(&B.empty[i], 1);
            mbar_init(&B.hand[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&B.rfull[i], 1);
            mbar_init(&B.rempty[i], kConvWarps + C::kScaleWarps);
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&B.cfull[i], 2);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&B.sfull[i], 1);
            mbar_init(&B.pfull[i], C::kGroups ? kSoftWarps / 2 : kSoftWarps);
        }
        mbar_init(&B.odone[0], 1);
        mbar_init(&B.odone[1], 1);
        mbar_init(&B.oend, 1);
        mbar_init(&B.ofree, kSoftWarps);
        mbar_init(&B.qfull, kSoftWarps);
        mbar_init(&B.drain, 1);
        fence_mbar_init();
        B.abort_flag = 0;
        B.odd = 0;
        for (int i = 0; i < kSoftWarps; ++i) B.gave_up[i] = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&B.tmem, 512);
    pdl_wait_previous();  // (before its dependents, which read the call's inputs at once)
    pdl_launch_dependents();
    tc_fence_before();
    const Share share = find_share<kTcRows, TN, C::kThreads>(a);  // (synchronises the CTA)
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);  // (warp-uniform to the compiler)
    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            set_status(a.status, kStatusTimeout);
        }
    };
    const int page = 1 << a.c.page_shift;
    const int run_shift = a.c.page_shift < 6 ? a.c.page_shift : 6;  // tokens of one page in a tile
    const int run = 1 << run_shift, runs = TN >> run_shift;
    static_assert(TN == 64, "run_shift");
    // bf16 tiles that the converters fill: with drafted tokens, or past the sequence's end
    auto by_hand = [&](const Segment& g, int tile) {
        return !E4M3 && (tile + 1) * TN > g.seq.len - g.seq.nodes;
    };
    Segment seg;
    bool have = first_segment<kTcRows, TN>(a, share, seg);
    bool ok = true;

    if (warp == kLoadWarp) {
        // ================================================================ loader
        if (!E4M3 && lane == 0) {
            prefetch_tmap(&map_k);
            prefetch_tmap(&map_v);
        }
        uint32_t last_full = 0, last_par = 0;    // copies in flight, for the end
        int rst = 0, rpar = 1;                   // raw slot, phase of its last release
        int st = 0, par = 1;                     // slot, likewise
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
            // This lane's page of a tile (every lane's, where a page holds a tile). The
            // table is read one tile ahead, and what is read is not looked at before
            // its tile comes.
            const int at = run == TN ? 0 : lane;
            const int32_t* table = a.p.table + (int64_t)seg.n * a.p.max_pages;
            auto page_id = [&](int tile) -> int {
                const int pos = tile * TN + at * run;
                return tile < seg.tile1 && at < runs && pos < seg.seq.len ? __ldg(table + (pos >> a.c.page_shift)) : 0;
            };
            int next_id = page_id(seg.tile0);
            for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile) {
                const int n_runs = (min(TN, seg.seq.len - tile * TN) + run - 1) >> run_shift;
                int id = next_id;
                next_id = page_id(tile + 1);
                if (id < 0 || id >= a.c.n_pages) {
                    set_status(a.status, kStatusBadSeqlens);
                    id = 0;  // some rows of the pool: the sequence's output means nothing
                }
                const int row = ((id * a.c.Hk + seg.hk) << a.c.page_shift) + ((tile * TN + at * run) & (page - 1));
                if (E4M3) {
                    if (!all_wait(&B.rempty[rst], rpar, abort_flag, wlim)) { ok = false; break; }
                    uint8_t* dst = sm + C::kOffRaw + rst * C::kRaw;
                    if (lane == 0) mbar_arrive_expect_tx(&B.rfull[rst], (uint32_t)(2 * n_runs * run * (D + 4)));
                    last_full |= 1u << rst;
                    last_par = (last_par & ~(1u << rst)) | (uint32_t)(rpar ^ 1) << rst;
                    __syncwarp();
                    if (lane < n_runs) {
                        const int at_row = lane * run;
                        bulk_load(dst + at_row * D, static_cast<const uint8_t*>(a.c.k) + (int64_t)row * D, run * D, &B.rfull[rst]);
                        bulk_load(dst + (TN + at_row) * D, static_cast<const uint8_t*>(a.c.v) + (int64_t)row * D, run * D,
                                  &B.rfull[rst]);
                        bulk_load(dst + 2 * TN * D + at_row * 4, a.c.k_scale + row, run * 4, &B.rfull[rst]);
                        bulk_load(dst + 2 * TN * D + (TN + at_row) * 4, a.c.v_scale + row, run * 4, &B.rfull[rst]);
                    }
                    __syncwarp();
                    if (++rst == C::kRawSlots) rst = 0, rpar ^= 1;
                } else {
                    if (!all_wait(&B.empty[st], par, abort_flag, wlim) || !all_wait(&B.empty[st + 1], par, abort_flag, wlim)) {
                        ok = false;
                        break;
                    }
                    if (by_hand(seg, tile)) {  // (the converters walk only these: the slots' phases are followed here)
                        // the last copy into this slot has landed (its products are done, or the slot
                        // would not be free), and the phase now begun is the converters'
                        last_full &= ~(1u << st);
                        if (lane == 0) mbar_arrive(&B.hand[st]);
                    } else {
                        uint8_t* dst = sm + st * C::kSlot;
                        last_full |= 1u << st;
                        last_par = (last_par & ~(1u << st)) | (uint32_t)(par ^ 1) << st;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&B.full[st], 2 * C::kSlot);
                            mbar_arrive(&B.full[st]);
                            if (run == TN) {
                                tma_load_3d(dst, &map_k, &B.full[st], 0, row, 0);
                                tma_load_3d(dst + C::kSlot, &map_v, &B.full[st], 0, row, 0);
                            }
                        }
                        __syncwarp();
                        if (run < TN && lane < runs) {
#pragma unroll
                            for (int b = 0; b < C::kBlocks; ++b) {
                                uint8_t* d = dst + b * C::kBlock + lane * run * 128;
                                tma_load_3d(d, &map_k, &B.full[st], 0, row, b);
                                tma_load_3d(d + C::kSlot, &map_v, &B.full[st], 0, row, b);
                            }
                        }
                        __syncwarp();
                    }
                    if ((st += 2) == C::kSlots) st = 0, par ^= 1;
                }
            }
        }
        if (!ok) fail();
        // no copy may land after the CTA is gone
        if (lane == 0)
            for (int x = 0; x < (E4M3 ? C::kRawSlots : C::kSlots); ++x)
                if ((last_full >> x) & 1 && !mbar_wait(E4M3 ? &B.rfull[x] : &B.full[x], (last_par >> x) & 1, kDrainWaitNs))
                    set_status(a.status, kStatusTimeout);
        __syncwarp();
    } else if (E4M3 && warp >= C::kScaleWarp0) {
        // ================================================================= scales
        // of keys (first warp) and of values, with their logarithms: two tokens a lane
        const int kv = warp - C::kScaleWarp0;
        int i = 0, rs = 0, rpar = 0, sl = 0;
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg))
            for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile, ++i) {
                if (!all_wait(&B.rfull[rs], rpar, abort_flag, wlim)) { ok = false; break; }
                const float2 raw = reinterpret_cast<const float2*>(sm + C::kOffRaw + rs * C::kRaw + 2 * TN * D)[kv * (TN / 2) + lane];
                const int left = seg.seq.len - tile * TN - 2 * lane;
                const float2 x = make_float2(left > 0 ? raw.x : 0.f, left > 1 ? raw.y : 0.f);
                float2* out = reinterpret_cast<float2*>(scales + sl * 3 * TN) + kv * (TN / 2) + lane;
                *out = x;
                if (kv) out[TN / 2] = make_float2(log2_scale(x.x), log2_scale(x.y));
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&B.cfull[sl]);
                    mbar_arrive(&B.rempty[rs]);
                }
                if (++rs == C::kRawSlots) rs = 0, rpar ^= 1;
                if (++sl == kScaleSlots) sl = 0;
            }
        if (!ok) fail();
    } else if (warp >= kConvWarp0) {
        // =================================================== conversion, last tiles
        static_assert(E4M3 || kConvWarps == 2, "a warp for keys and one for values");
        int rs = 0, rpar = 0, st = 0, par = 1;   // raw slot and slot of its keys, their phases
        uint32_t hand_par = 0;                   // per slot: phase of its next hand-over
        auto publish = [&](uint64_t* bar) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
            for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile) {
                const int left = seg.seq.len - tile * TN;  // tokens that exist, from the tile's first
                if (E4M3) {
                    if (!all_wait(&B.rfull[rs], rpar, abort_flag, wlim)) { ok = false; break; }
                    const uint8_t* raw = sm + C::kOffRaw + rs * C::kRaw;
                    // A lane takes 16-byte pieces of every second token: piece col of block
                    // y ^ h, h the token's parity. Eight lanes then read 64 bytes each of
                    // two rows, in different bank groups, and write two rows of two blocks
                    // whose swizzles fall into different bank groups as well. A batch of
                    // pieces is read before the one ahead of it is written.
                    constexpr int kBatch = C::kBlocks > 1 ? 4 : 2;          // pieces: two tokens of one or two blocks
                    constexpr int kSide = 2 * C::kBlocks / kBatch;          // batches of a tile's keys, or values
                    const int col = lane & 3, h = (lane >> 2) & 1;
                    const int tok0 = 8 * (warp - kConvWarp0) + 2 * (lane >> 3) + h;
                    const uint8_t* in = raw + tok0 * D + 16 * col;
                    uint8_t* const slot = sm + st * C::kSlot;
                    const uint32_t at0 = sw128_off(tok0, 2 * col), at1 = sw128_off(tok0, 2 * col + 1);
                    const bool whole = left >= TN;
                    uint4 u[2][kBatch];
                    auto block = [&](int b, int j) { return C::kBlocks > 1 ? (b % kSide * (kBatch / 2) + j / 2) ^ h : 0; };
                    auto load = [&](int b) {
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            u[b & 1][j] = *reinterpret_cast<const uint4*>(in + (b / kSide * TN + 32 * (j & 1)) * D + 64 * block(b, j));
                            if (!whole && tok0 + 32 * (j & 1) >= left) u[b & 1][j] = make_uint4(0, 0, 0, 0);
                        }
                    };
                    load(0);
#pragma unroll
                    for (int b = 0; b < 2 * kSide; ++b) {
                        if (b + 1 < 2 * kSide) load(b + 1);
                        if (b % kSide == 0) ok = ok && all_wait(&B.empty[st + b / kSide], par, abort_flag, wlim);
                        if (!ok) break;
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            uint8_t* out = slot + b / kSide * C::kSlot + block(b, j) * C::kBlock + 32 * (j & 1) * 128;
                            const uint4 x = u[b & 1][j];
                            *reinterpret_cast<uint4*>(out + at0) = make_uint4(e4m3x2_to_f16x2(x.x), e4m3x2_to_f16x2(x.x >> 16),
                                                                             e4m3x2_to_f16x2(x.y), e4m3x2_to_f16x2(x.y >> 16));
                            *reinterpret_cast<uint4*>(out + at1) = make_uint4(e4m3x2_to_f16x2(x.z), e4m3x2_to_f16x2(x.z >> 16),
                                                                             e4m3x2_to_f16x2(x.w), e4m3x2_to_f16x2(x.w >> 16));
                        }
                        if (b == 2 * kSide - 1) {  // (all pieces are in registers: the raw slot is free)
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&B.rempty[rs]);
                        }
                        if (!C::kOneFull && b % kSide == kSide - 1) publish(&B.full[st + b / kSide]);
                    }
                    if (!ok) break;
                    if (C::kOneFull) publish(&B.full[st]);
                    if (++rs == C::kRawSlots) rs = 0, rpar ^= 1;
                    if ((st += 2) == C::kSlots) st = 0, par ^= 1;
                } else {
                    if (by_hand(seg, tile)) {
                        const int kv = warp - kConvWarp0;  // a warp for keys, one for values
                        uint8_t* slot = sm + (st + kv) * C::kSlot;
                        if (!all_wait(&B.hand[st], (hand_par >> st) & 1, abort_flag, wlim)) { ok = false; break; }
                        hand_par ^= 1u << st;
                        constexpr int kPer = D / 8;
                        const int draft = seg.seq.len - seg.seq.nodes - tile * TN;  // the draft's first token here
                        bool odd = false;
#pragma unroll 4
                        for (int y = lane; y < TN * kPer; y += 32) {
                            const int tok = y / kPer, col = y % kPer;
                            uint4 u = make_uint4(0, 0, 0, 0);
                            if (tok < left) {
                                const int64_t row = page_row(a.p, a.c, seg.n, tile * TN + tok);
                                if (row < 0) set_status(a.status, kStatusBadSeqlens);
                                else
                                    u = *(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv ? a.c.v : a.c.k) +
                                                                         (row + ((int64_t)seg.hk << a.c.page_shift)) * D) + col);
                            }
                            if (kv && tok >= draft) {
                                odd |= zero_non_finite(u.x);
                                odd |= zero_non_finite(u.y);
                                odd |= zero_non_finite(u.z);
                                odd |= zero_non_finite(u.w);
                            }
                            *reinterpret_cast<uint4*>(slot + (col >> 3) * C::kBlock + sw128_off(tok, col & 7)) = u;
                        }
                        if (odd) *reinterpret_cast<volatile int*>(&B.odd) = 1;
                        publish(&B.full[st]);
                    }
                    if ((st += 2) == C::kSlots) st = 0;
                }
            }
        }
        if (!ok) fail();
    } else if (warp == kMmaWarp) {
        // ================================================================ products
        // The whole warp walks the tiles alike and one elected lane issues. The
        // products' operands live in uniform registers; where the compiler cannot
        // see that a value is the same in every lane it moves each of them there
        // before each product, which costs more than the product. Hence the
        // shuffles, and no way out of the loops but their counts: once a wait has
        // run out the rest is walked without issuing anything.
        const uint64_t kd = sw128_desc(smem_u32(sm), 16, 1024), vd = sw128_desc(smem_u32(sm), C::kBlock, 1024);
        int ks = 0, vs = 1, kpar = 0, vpar = 0;  // slots of the next keys and values, their phases
        int sb = 0, pb = 0, ppar = 0;            // buffers of the next scores and probabilities
        int og = 0;                              // accumulator of the next tile
        auto scores = [&]() {                    // S of the next tile
            ok = ok && all_wait(&B.full[ks], kpar, abort_flag, wlim);
            tc_fence_after();
            const uint64_t d0 = kd + (uint64_t)(ks * (C::kSlot >> 4));
            const uint32_t s0 = tmem + C::kColS + sb * TN;
            if (elect_one() && ok) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16_ta(s0, tmem + C::kColQ + 8 * kk, d0 + (((kk >> 2) * C::kBlock + 32 * (kk & 3)) >> 4), C::kIdescS,
                                kk > 0);
                mma_commit(&B.sfull[sb]);
                mma_commit(&B.empty[ks]);
            }
            __syncwarp();
            if ((ks += 2) >= C::kSlots) ks = 0, kpar ^= 1;
            if (++sb == C::kBufs) sb = 0;
        };
        bool more_segs = __shfl_sync(0xffffffffu, (int)have, 0);
        for (int seg_no = 0; more_segs; ++seg_no) {
            const int tiles = __shfl_sync(0xffffffffu, seg.tile1 - seg.tile0, 0);
            ok = ok && all_wait(&B.qfull, seg_no & 1, abort_flag, wlim);
            for (int y = 0; y < C::kBufs && y < tiles; ++y) scores();
            ok = ok && (seg_no == 0 || all_wait(&B.ofree, (seg_no - 1) & 1, abort_flag, wlim));
            for (int y = 0; y < tiles; ++y) {
                ok = ok && (C::kOneFull || all_wait(&B.full[vs], vpar, abort_flag, wlim)) &&
                     all_wait(&B.pfull[pb], ppar, abort_flag, wlim);
                tc_fence_after();
                const uint64_t d0 = vd + (uint64_t)(vs * (C::kSlot >> 4));
                const uint32_t p0 = tmem + C::kColS + pb * TN, o0 = tmem + (C::kGroups ? og * D : 0);
                const bool more = y >= (C::kGroups ? 2 : 1);  // the accumulator holds something
                if (elect_one() && ok) {
#pragma unroll
                    for (int kk = 0; kk < TN / 16; ++kk)
                        mma_bf16_ta(o0, p0 + 8 * kk, d0 + (2048 * kk >> 4), C::kIdescO, more || kk > 0);
                    mma_commit(&B.empty[vs]);
                    mma_commit(&B.odone[C::kGroups ? og : 0]);
                    if (y + 1 == tiles) mma_commit(&B.oend);
                }
                __syncwarp();
                if ((vs += 2) >= C::kSlots) vs = 1, vpar ^= 1;
                if (++pb == C::kBufs) pb = 0, ppar ^= 1;
                og ^= 1;
                // the buffer of these probabilities takes the scores kBufs tiles on
                if (y + C::kBufs < tiles) scores();
            }
            more_segs = __shfl_sync(0xffffffffu, (int)(next_segment<kTcRows, TN>(a, share, seg)), 0);
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) mma_commit(&B.drain);
        __syncwarp();
        if (!mbar_wait(&B.drain, 0, kDrainWaitNs)) set_status(a.status, kStatusTimeout);
    } else {
        // ================================================================= softmax
        const int quarter = warp & 3, half = warp >> 2;  // half: of the columns, or the group
        const int m = 32 * quarter + lane;               // row of the tile, lane of tensor memory
        const int pair = 1 + quarter;                    // named barrier of the two warps with the same rows
        const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
        int i = 0;  // tile number in this CTA
        for (int seg_no = 0; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg), ++seg_no) {
            const bool busy = 32 * quarter < seg.rows, live = m < seg.rows;
            const int r = seg.rt * kTcRows + (live ? m : 0);
            const int node = r / G, head = seg.hk * G + r % G;
            const int64_t t = seg.seq.first + node;
            const int base = seg.seq.len - seg.seq.nodes;
            uint64_t sees = 0;
            if (live) {
                sees = a.mask ? (uint64_t)a.mask[t] : (2ull << node) - 1;
                if (seg.seq.nodes < 64) sees &= (1ull << seg.seq.nodes) - 1;
            }
            float ref = kNegInf, mul = a.scale * kLog2e;
            float2 l2 = make_float2(0.f, 0.f);
            // ---- queries, half of the row per warp (every product that reads the last
            // segment's is done)
            if (busy) {
                const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + t * a.ld_q +
                                                                 (int64_t)head * D + half * (D / 2));
                uint4 u[D / 16];  // (all of it at once: nothing else hides the reads' latency here)
#pragma unroll
                for (int e = 0; e < D / 16; ++e) u[e] = live ? __ldg(qp + e) : make_uint4(0, 0, 0, 0);
                float down = 1.f;
                if (E4M3) {
                    // as f16, the row scaled by a power of two
                    uint32_t big = 0;
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) {
                        const uint32_t w[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) big = max(big, max(w[y] & 0x7FFFu, w[y] >> 16 & 0x7FFFu));
                    }
                    row_top[half * 128 + m] = __uint_as_float(big);
                    pair_sync(pair);
                    big = max(big, __float_as_uint(row_top[(half ^ 1) * 128 + m]));
                    float up;
                    query_scale(big, down, up);
                    mul *= up;
                }
#pragma unroll
                for (int c0 = 0; c0 < D / 2; c0 += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 x = u[c0 / 8 + e];
                        w[4 * e] = x.x; w[4 * e + 1] = x.y; w[4 * e + 2] = x.z; w[4 * e + 3] = x.w;
                    }
                    if (E4M3) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = pack_f16(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xFFFF0000u) * down);
                    }
                    tmem_st16(tmem + lane_off + C::kColQ + half * (D / 4) + c0 / 2, w);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.qfull);
            if (E4M3 && busy) pair_sync(pair);  // (what the warps told each other is read)

            const int tiles = seg.tile1 - seg.tile0, i1 = i + tiles;
            if constexpr (C::kGroups) {
                // ---- this group's tiles: scores in two passes of 32 columns at a time
                const int first = i + ((i ^ half) & 1);
                for (int x = first; x < i1; x += 2) {
                    const int tile = seg.tile0 + x - i;
                    ok = all_wait(&B.sfull[x % 3], (x / 3) & 1, abort_flag, wlim) &&
                         (!E4M3 || all_wait(&B.cfull[x % kScaleSlots], (x / kScaleSlots) & 1, abort_flag, wlim));
                    if (!ok) break;
                    tc_fence_after();
                    if (busy) {
                        const uint32_t s0 = tmem + lane_off + C::kColS + (x % 3) * TN;
                        const float* sc = scales + (x % kScaleSlots) * 3 * TN;
                        const int off = tile * TN - base;  // the tile's start past the context
                        auto softmax = [&](auto masked_) {
                            constexpr bool masked = decltype(masked_)::value;
                            const float2 mul_2 = make_float2(mul, mul);
                            float top = kNegInf, top_b = kNegInf;
                            // (e4m3: rolled, or its 128 registers do not hold it)
#pragma unroll(E4M3 ? 1 : 2)
                            for (int c0 = 0; c0 < TN; c0 += 32) {
                                float2 s[16];
                                tmem_ld32(s0 + c0, *reinterpret_cast<float(*)[32]>(&s[0]));
                                tmem_wait_ld();
                                if (E4M3) {  // scaled scores back to tensor memory; maxima are of the weights
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float4 k4 = *reinterpret_cast<const float4*>(sc + c0 + 2 * e);
                                        s[e] = mul2(s[e], mul2(mul_2, make_float2(k4.x, k4.y)));
                                        s[e + 1] = mul2(s[e + 1], mul2(mul_2, make_float2(k4.z, k4.w)));
                                    }
                                    tmem_st32(s0 + c0, *reinterpret_cast<const float(*)[32]>(&s[0]));
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float4 v4 = *reinterpret_cast<const float4*>(sc + 2 * TN + c0 + 2 * e);
                                        s[e] = add2(s[e], make_float2(v4.x, v4.y));
                                        s[e + 1] = add2(s[e + 1], make_float2(v4.z, v4.w));
                                    }
                                }
                                if (masked) {
                                    const uint32_t bits = sees32(sees, off + c0);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        if (!((bits >> (2 * e)) & 1)) s[e].x = kNegInf;
                                        if (!((bits >> (2 * e + 1)) & 1)) s[e].y = kNegInf;
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    top = max3(top, s[e].x, s[e].y);
                                    top_b = max3(top_b, s[e + 1].x, s[e + 1].y);
                                }
                            }
                            top = fmaxf(top, top_b);
                            if (!E4M3) top *= mul;  // (the scale is positive)
                            // ---- the reference: moved when outgrown
                            const bool move = top > ref + (kLazy + kLift<E4M3>);
                            if (__any_sync(0xffffffffu, move)) {
                                top -= kLift<E4M3>;
                                const float f = move && ref != kNegInf ? exp2_approx(ref - top) : 1.f;
                                if (move) ref = top;
                                if (x != first && __any_sync(0xffffffffu, f != 1.f)) {
                                    l2 = mul2(l2, make_float2(f, f));
                                    // the group's last output product (the scores of its tile before
                                    // are complete, and with them the one before that)
                                    if (!all_wait(&B.odone[half], ((x >> 1) - 1) & 1, abort_flag, wlim)) ok = false;
                                    tc_fence_after();
#pragma unroll 1
                                    for (int c0 = 0; c0 < D; c0 += 32) {
                                        float o[32];
                                        tmem_ld32(tmem + lane_off + half * D + c0, o);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int e = 0; e < 32; ++e) o[e] *= f;
                                        tmem_st32(tmem + lane_off + half * D + c0, o);
                                    }
                                    tmem_wait_st();
                                }
                            }
                            const float minus = ref == kNegInf ? 0.f : -ref;
                            const float2 minus_2 = make_float2(minus, minus);
                            if (E4M3) tmem_wait_st();
#pragma unroll(E4M3 ? 1 : 2)
                            for (int c0 = 0; c0 < TN; c0 += 32) {
                                float2 s[16];
                                tmem_ld32(s0 + c0, *reinterpret_cast<float(*)[32]>(&s[0]));
                                tmem_wait_ld();
                                const uint32_t bits = masked ? sees32(sees, off + c0) : 0xFFFFFFFFu;
                                uint32_t p[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float2 y = E4M3 ? add2(s[e], minus_2) : fma2(s[e], mul_2, minus_2);
                                    y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                    if (masked) {  // nothing from a token that the row does not see
                                        if (!((bits >> (2 * e)) & 1)) y.x = 0.f;
                                        if (!((bits >> (2 * e + 1)) & 1)) y.y = 0.f;
                                    }
                                    l2 = add2(l2, y);
                                    if (!E4M3) p[e] = pack_bf16(y.x, y.y);
                                    else s[e] = y;
                                }
                                if (E4M3) {
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float4 v4 = *reinterpret_cast<const float4*>(sc + TN + c0 + 2 * e);
                                        s[e] = mul2(s[e], make_float2(v4.x, v4.y));
                                        s[e + 1] = mul2(s[e + 1], make_float2(v4.z, v4.w));
                                    }
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        if (masked) {  // (whatever its scale)
                                            if (!((bits >> (2 * e)) & 1)) s[e].x = 0.f;
                                            if (!((bits >> (2 * e + 1)) & 1)) s[e].y = 0.f;
                                        }
                                        p[e] = pack_f16(s[e].x, s[e].y);
                                    }
                                }
                                tmem_st16(s0 + c0 / 2, p);
                            }
                            tmem_wait_st();
                        };
                        if (off + TN > 0) softmax(Bool<true>{});
                        else softmax(Bool<false>{});
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B.pfull[x % 3]);
                    if (!ok) break;
                }
            } else {
                // ---- half of every tile's columns
                constexpr int HC = TN / 2;
                for (int x = i; x < i1; ++x) {
                    const int tile = seg.tile0 + x - i, b = x & 1;
                    // A warp whose wait runs out goes on to the vote below, where its partner
                    // learns of it: neither may stay alone at their barrier.
                    ok = all_wait(&B.sfull[b], (x >> 1) & 1, abort_flag, wlim) &&
                         (!E4M3 || all_wait(&B.cfull[x % kScaleSlots], (x / kScaleSlots) & 1, abort_flag, wlim)) && ok;
                    tc_fence_after();
                    if (busy) {
                        const uint32_t s0 = tmem + lane_off + C::kColS + b * TN;
                        const float* sc = scales + (x % kScaleSlots) * 3 * TN + half * HC;
                        const int off = tile * TN + half * HC - base;  // this half's start past the context
                        const bool masked = off + HC > 0;
                        const uint32_t bits = masked ? sees32(sees, off) : 0xFFFFFFFFu;
                        static_assert(HC == 32 || C::kGroups, "one load per half");
                        float2 s[16];
                        tmem_ld32(s0 + half * HC, *reinterpret_cast<float(*)[32]>(&s[0]));
                        tmem_wait_ld();
                        const float2 mul_2 = make_float2(mul, mul);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float2 k2 = mul_2, k3 = mul_2;
                            if (E4M3) {
                                const float4 k4 = *reinterpret_cast<const float4*>(sc + 2 * e);
                                k2 = mul2(mul_2, make_float2(k4.x, k4.y));
                                k3 = mul2(mul_2, make_float2(k4.z, k4.w));
                            }
                            s[e] = mul2(s[e], k2);
                            s[e + 1] = mul2(s[e + 1], k3);
                        }
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                if (!((bits >> (2 * e)) & 1)) s[e].x = kNegInf;
                                if (!((bits >> (2 * e + 1)) & 1)) s[e].y = kNegInf;
                            }
                        }
                        float top = kNegInf, top_b = kNegInf;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float2 y = s[e], z = s[e + 1];
                            if (E4M3) {
                                const float4 v4 = *reinterpret_cast<const float4*>(sc + 2 * TN + 2 * e);
                                y = add2(y, make_float2(v4.x, v4.y));
                                z = add2(z, make_float2(v4.z, v4.w));
                            }
                            top = max3(top, y.x, y.y);
                            top_b = max3(top_b, z.x, z.y);
                        }
                        top = fmaxf(top, top_b);
                        // ---- the reference: moved when either half outgrows it (both warps have
                        // read their scores when the vote is out: probabilities may overwrite them)
                        if (pair_any(pair, !ok || (live && top > ref + (kLazy + kLift<E4M3>)))) {
                            row_top[half * 128 + m] = top;
                            if (!ok) B.gave_up[warp] = 1;
                            pair_sync(pair);
                            ok = ok && !B.gave_up[warp ^ 4];
                            if (!ok) break;
                            top = fmaxf(top, row_top[(half ^ 1) * 128 + m]) - kLift<E4M3>;
                            const bool move = top > ref;
                            const float f = move && ref != kNegInf ? exp2_approx(ref - top) : 1.f;
                            if (move) ref = top;
                            l2 = mul2(l2, make_float2(f, f));
                            if (x != i) {
                                if (!all_wait(&B.odone[0], (x - 1) & 1, abort_flag, wlim)) ok = false;
                                tc_fence_after();
#pragma unroll 1
                                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                                    float o[32];
                                    tmem_ld32(tmem + lane_off + c0, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] *= f;
                                    tmem_st32(tmem + lane_off + c0, o);
                                }
                                tmem_wait_st();
                            }
                            pair_sync(pair);  // the maxima are read
                        }
                        const float minus = ref == kNegInf ? 0.f : -ref;
                        const float2 minus_2 = make_float2(minus, minus);
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            s[e] = add2(s[e], minus_2);
                            s[e] = make_float2(exp2_approx(s[e].x), exp2_approx(s[e].y));
                            l2 = add2(l2, s[e]);
                        }
                        if (E4M3) {
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float4 v4 = *reinterpret_cast<const float4*>(sc + TN + 2 * e);
                                s[e] = mul2(s[e], make_float2(v4.x, v4.y));
                                s[e + 1] = mul2(s[e + 1], make_float2(v4.z, v4.w));
                            }
                            if (masked) {  // nothing from a token that the row does not see, whatever its scale
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    if (!((bits >> (2 * e)) & 1)) s[e].x = 0.f;
                                    if (!((bits >> (2 * e + 1)) & 1)) s[e].y = 0.f;
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = E4M3 ? pack_f16(s[e].x, s[e].y) : pack_bf16(s[e].x, s[e].y);
                        tmem_st16(s0 + half * HC / 2, p);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B.pfull[b]);
                    if (!busy && !ok) break;
                }
            }
            // ---- the segment's output
            const int i0 = i;
            i = i1;
            ok = ok && all_wait(&B.oend, seg_no & 1, abort_flag, wlim);
            if (busy ? pair_any(pair, !ok) : !ok) { ok = false; break; }
            tc_fence_after();
            const bool odd = !E4M3 && *reinterpret_cast<volatile int*>(&B.odd) != 0;
            if (busy) {
                row_top[half * 128 + m] = ref;
                row_sum[half * 128 + m] = l2.x + l2.y;
                pair_sync(pair);
                // the two sums under one reference; a group without a tile has no output
                const float ref_0 = row_top[m], ref_1 = row_top[128 + m];
                float l = 0.f, f_0 = 1.f, f_1 = 1.f;
                if (C::kGroups) {
                    ref = fmaxf(ref_0, ref_1);
                    f_0 = ref_0 == kNegInf ? 1.f : exp2_approx(ref_0 - ref);  // (nothing but zeros, or NaN)
                    f_1 = ref_1 == kNegInf ? 1.f : exp2_approx(ref_1 - ref);
                }
                l = row_sum[m] * f_0 + row_sum[128 + m] * f_1;
                const bool have_0 = !C::kGroups || tiles > 1 || !(i0 & 1), have_1 = C::kGroups && (tiles > 1 || (i0 & 1));
                const bool whole = seg.whole();
                if (tid == 0) note_parts(a, seg);
                const bool empty = ref == kNegInf && l == 0.f;
                const float inv = empty ? 0.f : 1.f / l;
                const int64_t out = (t * a.H + head) * D;
                float* part = partial_base(a) + (2 * (int64_t)blockIdx.x + seg.later) * slot_floats(D, a.slot_rows);
                if (!whole && live && half == 0) {
                    part[m] = ref;
                    part[a.slot_rows + m] = l;
                }
                part += 2 * a.slot_rows + m * D;
#pragma unroll 1
                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                    float o[32];
                    if (have_0) {
                        tmem_ld32(tmem + lane_off + c0, o);
                        tmem_wait_ld();
                    }
                    if (C::kGroups) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = have_0 ? o[e] * f_0 : 0.f;
                        if (have_1) {
                            float o1[32];
                            tmem_ld32(tmem + lane_off + D + c0, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], f_1, o[e]);
                        }
                    }
                    if (!live) continue;
                    if (odd) {
                        // drafted values that are not finite, for the rows that see them
                        const int from = max(base, seg.tile0 * TN), to = min(seg.seq.len, seg.tile1 * TN);
                        for (int p = from; p < to; ++p) {
                            if (!((sees >> (p - base)) & 1)) continue;
                            const int64_t vr = page_row(a.p, a.c, seg.n, p);
                            if (vr < 0) continue;
                            const uint16_t* v = static_cast<const uint16_t*>(a.c.v) +
                                                (vr + ((int64_t)seg.hk << a.c.page_shift)) * D + c0;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float y = bf16_to_f32(v[e]);
                                if (!(fabsf(y) <= FLT_MAX)) o[e] += y;
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
                if (whole && live && half == 0 && a.lse)
                    a.lse[t * a.H + head] = empty ? kNegInf : ref * kLn2 + logf(l);
                pair_sync(pair);  // what the warps told each other is read
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The cache's rows [n_pages * Hk * page, D] bf16 as (64 elements, row, block of 64
// elements); boxes of the rows of a page that one tile can take, 128-byte
// swizzle: all blocks at once where that is the whole tile, else one.
bool make_map(CUtensorMap* m, const void* ptr, const CacheView& c, int rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)((c.n_pages * c.Hk) << c.page_shift), (cuuint64_t)(c.D / 64)};
    cuuint64_t strides[2] = {(cuuint64_t)c.D * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)rows, rows == TN ? (cuuint32_t)(c.D / 64) : 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3>
cudaError_t launch_tc(const TreeArgs& a, cudaStream_t s) {
    using C = Tc<D, E4M3>;
    CUtensorMap mk = {}, mv = {};
    const int page = 1 << a.c.page_shift, run = page < TN ? page : TN;
    if (!E4M3 && (!make_map(&mk, a.c.k, a.c, run) || !make_map(&mv, a.c.v, a.c, run))) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_tc_kernel<D, E4M3>, dim3(a.grid), dim3(C::kThreads), C::kSmem, s, a, mk, mv);
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
