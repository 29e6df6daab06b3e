// Attention of a drafted tree over the paged cache, on the tensor cores' tcgen05
// path (formula in tree_attn.cu): more than 16 query rows of a key/value head.
//
// A unit is (sequence, key/value head, 128 query rows), rows the M side of the
// products. One persistent CTA per SM walks an equal share of its row tile's
// line in tiles of TN tokens; 14 warps:
//   warps 0-7    softmax: two warps per 32 rows, half of the tile's tokens each,
//                a row per thread; probabilities back to tensor memory; the
//                output at the end of a segment
//   warp 8       issues the products: S = Q K^T of tile i + 1 goes out before
//                O += P V of tile i, so that the next scores form meanwhile
//   warp 9       loader: the tile's pages, a lane per page. bf16 tiles go
//                straight to their slots by TMA (128-byte swizzle); e4m3 pages
//                by bulk copies into a raw ring
//   warps 10-13  e4m3: raw tiles to f16 (exact) in the layout of the products;
//                bf16: the tiles that hold drafted tokens or end the sequence,
//                where rows past its end and drafted values that are not finite
//                must be zero
// Queries and probabilities are the products' A operands in tensor memory, so
// that shared memory -- written by the copies, read and written by the
// conversion, read by the products -- carries only the tiles.
// Tiles stand in one ring of slots in the order K0, V0, K1, V1, ..., so that the
// keys of the next tiles do not wait for the values of this one.
//
// Scales, f16 and the reference R are those of tree_attn.cu. Two warps share a
// row's reference: they vote at a named barrier on whether it has to move, and
// only then exchange maxima and rescale the output in tensor memory.
//
// Every wait is bounded (gdn_set_wait_limit_ns).
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

constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kConvWarp0 = 10, kConvWarps = 4;
constexpr int kTcThreads = 32 * (kConvWarp0 + kConvWarps), kConvThreads = 32 * kConvWarps;
constexpr int kScaleSlots = 4;
constexpr uint64_t kDrainWaitNs = 1000000000ull;

template <int D, bool E4M3>
struct Tc {
    static constexpr int TN = D == 256 ? 64 : 128;  // tokens of a tile
    static constexpr int kBlock = TN * 128;         // 64 elements of every row, 128-byte swizzled
    static constexpr int kBlocks = D / 64;
    static constexpr int kSlot = kBlock * kBlocks;
    static constexpr int kSlots = E4M3 ? 5 : 7;
    // raw e4m3 tiles: TN rows of D bytes, then TN scales
    static constexpr int kRaw = TN * D + TN * 4, kRawSlots = 3;
    static constexpr int kOffRaw = kSlots * kSlot;
    static constexpr int kOffScale = kOffRaw + (E4M3 ? kRawSlots * kRaw : 0);  // [slot][k, v, log2 v][TN]
    static constexpr int kScaleBytes = E4M3 ? kScaleSlots * 3 * TN * 4 : 0;
    static constexpr int kOffRows = kOffScale + kScaleBytes;      // what two warps tell each other: [2][128]
    static constexpr int kOffBars = kOffRows + 2 * 128 * 4;
    static constexpr int kUsed = kOffBars + 368 + 1024;           // 1024: alignment
    // above half of the SM's shared memory, so that a CTA has its tensor memory to itself
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem + 512 <= 227 * 1024, "shared memory");
    // tensor memory: O, the queries, two buffers of S
    static constexpr int kColQ = D, kColS = D + D / 2;
    static constexpr uint32_t kFormat = E4M3 ? ~((1u << 7) | (1u << 10)) : ~0u;  // f16 operands: format bits 0
    static constexpr uint32_t kIdescS = idesc_bf16(128, TN, 0, 0) & kFormat;
    static constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1) & kFormat;
};

struct TcBars {
    uint64_t full[7], empty[7];      // slots of the products (4 converter warps, bf16: and the loader / commit)
    uint64_t rfull[3], rempty[3];    // raw slots (bulk copies / 4 warps)
    uint64_t hand[7];                // bf16: slot left to the converters (loader)
    uint64_t sfull[2], pfull[2];     // scores (commit), probabilities (8 warps)
    uint64_t odone, ofree;           // output product (commit), output read (8 warps)
    uint64_t qfull;                  // queries in tensor memory (8 warps)
    uint64_t cfull[kScaleSlots];     // a tile's scales (4 warps)
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int odd;                         // some drafted value was not finite
    int gave_up[kSoftWarps];         // a softmax warp whose wait ran out, for its partner
};
static_assert(sizeof(TcBars) <= 368, "barrier block");

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
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
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

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTcThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v) {
    using C = Tc<D, E4M3>;
    constexpr int TN = C::TN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TcBars& B = *reinterpret_cast<TcBars*>(sm + C::kOffBars);
    volatile int* abort_flag = &B.abort_flag;
    float* scales = reinterpret_cast<float*>(sm + C::kOffScale);
    float* row_top = reinterpret_cast<float*>(sm + C::kOffRows);  // [half][row]
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (warp-uniform to the compiler)
    const int G = a.H / a.c.Hk;
    const uint64_t wlim = a.wait_ns;
    pdl_launch_dependents();

    if (tid == 0) {
        for (int i = 0; i < 7; ++i) {
            mbar_init(&B.full[i], E4M3 ? kConvWarps : kConvWarps + 1);
            mbar_init(&B.empty[i], 1);
            mbar_init(&B.hand[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&B.rfull[i], 1);
            mbar_init(&B.rempty[i], kConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.sfull[i], 1);
            mbar_init(&B.pfull[i], kSoftWarps);
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&B.cfull[i], kConvWarps);
        mbar_init(&B.odone, 1);
        mbar_init(&B.ofree, kSoftWarps);
        mbar_init(&B.qfull, kSoftWarps);
        mbar_init(&B.drain, 1);
        fence_mbar_init();
        B.abort_flag = 0;
        B.odd = 0;
        for (int i = 0; i < kSoftWarps; ++i) B.gave_up[i] = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&B.tmem, 512);
    tc_fence_before();
    const Share share = find_share<kTcRows, TN, kTcThreads>(a);  // (synchronises the CTA)
    tc_fence_after();
    const uint32_t tmem = B.tmem;
    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            set_status(a.status, kStatusTimeout);
        }
    };
    const int page = 1 << a.c.page_shift;
    const int run = page < TN ? page : TN;  // tokens of one page in a tile
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
        int x = 0;                               // group: tile x / 2's keys (even) or values
        uint32_t last_full = 0, last_par = 0;    // copies in flight, for the end
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
            for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile) {
                // this lane's page of the tile
                const int pos = tile * TN + lane * run;
                const int n_runs = min(TN / run, (min(TN, seg.seq.len - tile * TN) + run - 1) / run);
                int row = 0;
                if (lane < n_runs) {
                    row = (int)page_row(a.p, a.c, seg.n, pos);
                    if (row < 0) {
                        set_status(a.status, kStatusBadSeqlens);
                        row = 0;  // some rows of the pool: the sequence's output means nothing
                    } else {
                        row += seg.hk << a.c.page_shift;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++x) {
                    if (E4M3) {
                        const int st = x % C::kRawSlots, use = x / C::kRawSlots;
                        if (!all_wait(&B.rempty[st], (use & 1) ^ 1, abort_flag, wlim)) { ok = false; break; }
                        uint8_t* dst = sm + C::kOffRaw + st * C::kRaw;
                        if (lane == 0) mbar_arrive_expect_tx(&B.rfull[st], (uint32_t)(n_runs * run * (D + 4)));
                        last_full |= 1u << st;
                        last_par = (last_par & ~(1u << st)) | (uint32_t)(use & 1) << st;
                        __syncwarp();
                        if (lane < n_runs) {
                            bulk_load(dst + lane * run * D, static_cast<const uint8_t*>(kv ? a.c.v : a.c.k) + (int64_t)row * D,
                                      run * D, &B.rfull[st]);
                            bulk_load(dst + TN * D + lane * run * 4, (kv ? a.c.v_scale : a.c.k_scale) + row, run * 4,
                                      &B.rfull[st]);
                        }
                    } else {
                        const int st = x % C::kSlots, use = x / C::kSlots;
                        if (!all_wait(&B.empty[st], (use & 1) ^ 1, abort_flag, wlim)) { ok = false; break; }
                        if (by_hand(seg, tile)) {  // (the converters walk only these: a slot's phases are followed here)
                            if (lane == 0) {
                                mbar_arrive(&B.full[st]);
                                mbar_arrive(&B.hand[st]);
                            }
                            continue;
                        }
                        uint8_t* dst = sm + st * C::kSlot + lane * run * 128;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&B.full[st], C::kSlot);
                            mbar_arrive_n(&B.full[st], kConvWarps);
                        }
                        last_full |= 1u << st;
                        last_par = (last_par & ~(1u << st)) | (uint32_t)(use & 1) << st;
                        __syncwarp();
                        if (lane < n_runs) {
#pragma unroll
                            for (int b = 0; b < C::kBlocks; ++b)
                                tma_load_2d(dst + b * C::kBlock, kv ? &map_v : &map_k, &B.full[st], 64 * b, row);
                        }
                    }
                }
            }
        }
        if (!ok) fail();
        // no copy may land after the CTA is gone
        if (lane == 0)
            for (int st = 0; st < 7; ++st)
                if ((last_full >> st) & 1)
                    mbar_wait(E4M3 ? &B.rfull[st < 3 ? st : 0] : &B.full[st], (last_par >> st) & 1, kDrainWaitNs);
        __syncwarp();
    } else if (warp >= kConvWarp0) {
        // =================================================== conversion, last tiles
        const int pt = tid - 32 * kConvWarp0;
        int x = 0;
        uint32_t hand_par = 0;  // per slot: phase of its next hand-over
        auto publish = [&](uint64_t* bar) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
            for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile) {
                const int left = seg.seq.len - tile * TN;  // tokens that exist, from the tile's first
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++x) {
                    const int st = x % C::kSlots;
                    uint8_t* slot = sm + st * C::kSlot;
                    if (E4M3) {
                        const int rs = x % C::kRawSlots;
                        if (!all_wait(&B.rfull[rs], (x / C::kRawSlots) & 1, abort_flag, wlim)) { ok = false; break; }
                        const uint8_t* raw = sm + C::kOffRaw + rs * C::kRaw;
                        if (pt < TN) {
                            const float s = reinterpret_cast<const float*>(raw + TN * D)[pt];
                            float* out = scales + ((x >> 1) % kScaleSlots) * 3 * TN;
                            out[kv * TN + pt] = pt < left ? s : 0.f;
                            if (kv) out[2 * TN + pt] = log2_scale(pt < left ? s : 0.f);
                        }
                        if (kv) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&B.cfull[(x >> 1) % kScaleSlots]);
                        }
                        if (!all_wait(&B.empty[st], ((x / C::kSlots) & 1) ^ 1, abort_flag, wlim)) { ok = false; break; }
                        // A lane takes 16-byte pieces of every second token: piece col of block
                        // y ^ h, h the token's parity. Eight lanes then read 64 bytes each of
                        // two rows, in different bank groups, and write two rows of two blocks
                        // whose swizzles fall into different bank groups as well.
                        const int col = lane & 3, h = (lane >> 2) & 1;
                        const int tok0 = 8 * (warp - kConvWarp0) + 2 * (lane >> 3) + h;
                        const uint8_t* in = raw + tok0 * D + 16 * col;
                        uint8_t* out0 = slot + sw128_off(tok0, 2 * col);
                        uint8_t* out1 = slot + sw128_off(tok0, 2 * col + 1);
                        const bool whole = left >= TN;
#pragma unroll
                        for (int y = 0; y < C::kBlocks; ++y) {
                            const int block = C::kBlocks > 1 ? y ^ h : 0;
#pragma unroll
                            for (int j0 = 0; j0 < TN; j0 += 64) {
                                uint4 u[2];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    u[j] = *reinterpret_cast<const uint4*>(in + (j0 + 32 * j) * D + 64 * block);
                                    if (!whole && tok0 + j0 + 32 * j >= left) u[j] = make_uint4(0, 0, 0, 0);
                                }
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int at = block * C::kBlock + (j0 + 32 * j) * 128;
                                    *reinterpret_cast<uint4*>(out0 + at) =
                                        make_uint4(e4m3x2_to_f16x2(u[j].x), e4m3x2_to_f16x2(u[j].x >> 16),
                                                   e4m3x2_to_f16x2(u[j].y), e4m3x2_to_f16x2(u[j].y >> 16));
                                    *reinterpret_cast<uint4*>(out1 + at) =
                                        make_uint4(e4m3x2_to_f16x2(u[j].z), e4m3x2_to_f16x2(u[j].z >> 16),
                                                   e4m3x2_to_f16x2(u[j].w), e4m3x2_to_f16x2(u[j].w >> 16));
                                }
                            }
                        }
                        publish(&B.full[st]);
                        if (lane == 0) mbar_arrive(&B.rempty[rs]);  // (publish has synchronised the warp)
                    } else {
                        if (!by_hand(seg, tile)) continue;
                        if (!all_wait(&B.hand[st], (hand_par >> st) & 1, abort_flag, wlim)) { ok = false; break; }
                        hand_par ^= 1u << st;
                        constexpr int kPer = D / 8;
                        const int draft = seg.seq.len - seg.seq.nodes - tile * TN;  // the draft's first token here
                        bool odd = false;
#pragma unroll 2
                        for (int y = pt; y < TN * kPer; y += kConvThreads) {
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
                }
            }
        }
        if (!ok) fail();
    } else if (warp == kMmaWarp) {
        // ================================================================ products
        // The whole warp walks the tiles alike and one elected lane issues: the
        // descriptors are then warp-uniform values.
        // Descriptors of the ring's first slot; a slot, a block or a k-step further
        // is a constant added to the address field.
        const uint64_t kd = sw128_desc(smem_u32(sm), 16, 1024), vd = sw128_desc(smem_u32(sm), C::kBlock, 1024);
        int ks = 0, vs = 1, kpar = 0, vpar = 0;  // slots of the next keys and values, their phases
        auto advance = [](int& st, int& par) {   // two groups further
            st += 2;
            if (st >= C::kSlots) {
                st -= C::kSlots;
                par ^= 1;
            }
        };
        auto scores = [&](int b) -> bool {  // S of the next tile into buffer b
            if (!all_wait(&B.full[ks], kpar, abort_flag, wlim)) return false;
            tc_fence_after();
            const uint64_t d0 = kd + (uint64_t)(ks * (C::kSlot >> 4));
            const uint32_t s0 = tmem + C::kColS + b * TN;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16_ta(s0, tmem + C::kColQ + 8 * kk, d0 + (((kk >> 2) * C::kBlock + 32 * (kk & 3)) >> 4), C::kIdescS,
                                kk > 0);
                mma_commit(&B.sfull[b]);
                mma_commit(&B.empty[ks]);
            }
            __syncwarp();
            advance(ks, kpar);
            return true;
        };
        int b = 0, ppar = 0;
        if (have) ok = all_wait(&B.qfull, 0, abort_flag, wlim) && scores(0);
        for (int seg_no = 0; ok && have; ++seg_no) {
            const int tiles = seg.tile1 - seg.tile0;
            const bool more = next_segment<kTcRows, TN>(a, share, seg);
            if (seg_no > 0) ok = all_wait(&B.ofree, (seg_no - 1) & 1, abort_flag, wlim);
            for (int y = 0; ok && y < tiles; ++y) {
                // the next scores first: of this segment, or (below) of the next one
                if (y + 1 < tiles && !scores(b ^ 1)) { ok = false; break; }
                if (!all_wait(&B.full[vs], vpar, abort_flag, wlim) || !all_wait(&B.pfull[b], ppar, abort_flag, wlim)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t d0 = vd + (uint64_t)(vs * (C::kSlot >> 4));
                const uint32_t p0 = tmem + C::kColS + b * TN;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < TN / 16; ++kk)
                        mma_bf16_ta(tmem, p0 + 8 * kk, d0 + (2048 * kk >> 4), C::kIdescO, y > 0 || kk > 0);
                    mma_commit(&B.odone);
                    mma_commit(&B.empty[vs]);
                }
                __syncwarp();
                advance(vs, vpar);
                b ^= 1;
                if (b == 0) ppar ^= 1;
            }
            if (ok && more) ok = all_wait(&B.qfull, (seg_no + 1) & 1, abort_flag, wlim) && scores(b);
            have = more;
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) mma_commit(&B.drain);
        __syncwarp();
        mbar_wait(&B.drain, 0, kDrainWaitNs);
    } else {
        // ================================================================= softmax
        constexpr int HC = TN / 2;  // tokens of this warp's half
        const int quarter = warp & 3, half = warp >> 2;
        const int m = 32 * quarter + lane;  // row of the tile, lane of tensor memory
        const int pair = 1 + quarter;       // named barrier of the two warps
        const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
        int i = 0;
        for (; ok && have; have = ok && next_segment<kTcRows, TN>(a, share, seg)) {
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
            // ---- queries to tensor memory: half of the row per warp (the products that read
            // the last segment's are done: their scores have been here)
            if (busy) {
                const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + t * a.ld_q +
                                                                 (int64_t)head * D + half * (D / 2));
                float down = 1.f;
                if (E4M3) {
                    // as f16, the row scaled by a power of two that puts its largest element in [1, 2)
                    uint32_t big = 0;
#pragma unroll 4
                    for (int e = 0; e < D / 16; ++e) {
                        const uint4 u = live ? qp[e] : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) big = max(big, max(w[y] & 0x7FFFu, w[y] >> 16 & 0x7FFFu));
                    }
                    row_top[half * 128 + m] = __uint_as_float(big);
                    pair_sync(pair);
                    big = max(big, __float_as_uint(row_top[(half ^ 1) * 128 + m]));
                    uint32_t ex = big >> 7;  // a row that is not finite stays as it is
                    ex = ex == 255u || big == 0u ? 127u : ex < 1u ? 1u : ex > 253u ? 253u : ex;
                    down = __uint_as_float((254u - ex) << 23);
                    mul *= __uint_as_float(ex << 23);
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D / 2; c0 += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 u = live ? qp[c0 / 8 + e] : make_uint4(0, 0, 0, 0);
                        w[4 * e] = u.x; w[4 * e + 1] = u.y; w[4 * e + 2] = u.z; w[4 * e + 3] = u.w;
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
            for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++i) {
                const int b = i & 1;
                // A warp whose wait runs out goes on to the vote below, where its partner
                // learns of it: neither may stay alone at their barrier.
                ok = all_wait(&B.sfull[b], (i >> 1) & 1, abort_flag, wlim) &&
                     (!E4M3 || all_wait(&B.cfull[i % kScaleSlots], (i / kScaleSlots) & 1, abort_flag, wlim)) && ok;
                tc_fence_after();
                if (busy) {
                    const uint32_t s0 = tmem + lane_off + C::kColS + b * TN;
                    const float* sc = scales + (i % kScaleSlots) * 3 * TN + half * HC;
                    const int off = tile * TN + half * HC - base;  // this half's start past the context
                    const bool masked = off + HC > 0;
                    float2 s[HC / 2];
#pragma unroll
                    for (int c0 = 0; c0 < HC; c0 += 32)
                        tmem_ld32(s0 + half * HC + c0, *reinterpret_cast<float(*)[32]>(&s[c0 / 2]));
                    tmem_wait_ld();
                    const float2 mul_2 = make_float2(mul, mul);
                    if (E4M3) {
#pragma unroll
                        for (int e = 0; e < HC / 2; e += 2) {
                            const float4 k4 = *reinterpret_cast<const float4*>(sc + 2 * e);
                            s[e] = mul2(s[e], mul2(mul_2, make_float2(k4.x, k4.y)));
                            s[e + 1] = mul2(s[e + 1], mul2(mul_2, make_float2(k4.z, k4.w)));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < HC / 2; ++e) s[e] = mul2(s[e], mul_2);
                    }
                    if (masked) {
#pragma unroll
                        for (int c0 = 0; c0 < HC; c0 += 32) {
                            const uint32_t bits = sees32(sees, off + c0);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                if (!((bits >> (2 * e)) & 1)) s[c0 / 2 + e].x = kNegInf;
                                if (!((bits >> (2 * e + 1)) & 1)) s[c0 / 2 + e].y = kNegInf;
                            }
                        }
                    }
                    float top = kNegInf, top_b = kNegInf;
#pragma unroll
                    for (int e = 0; e < HC / 2; e += 2) {
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
                    if (pair_any(pair, !ok || (live && top > ref + kLazy))) {
                        row_top[half * 128 + m] = top;
                        if (!ok) B.gave_up[warp] = 1;
                        pair_sync(pair);
                        ok = ok && !B.gave_up[warp ^ 4];
                        if (!ok) break;
                        top = fmaxf(top, row_top[(half ^ 1) * 128 + m]);
                        const bool move = top > ref;
                        const float f = move && ref != kNegInf ? exp2_approx(ref - top) : 1.f;
                        if (move) ref = top;
                        l2 = mul2(l2, make_float2(f, f));
                        if (tile != seg.tile0) {
                            if (!all_wait(&B.odone, (i - 1) & 1, abort_flag, wlim)) ok = false;
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
#pragma unroll
                    for (int c0 = 0; c0 < HC; c0 += 32) {
                        const uint32_t bits = E4M3 && masked ? sees32(sees, off + c0) : 0xFFFFFFFFu;
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float2 y = add2(s[c0 / 2 + e], minus_2), z = add2(s[c0 / 2 + e + 1], minus_2);
                            y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            z = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                            l2 = add2(l2, add2(y, z));
                            if (E4M3) {
                                const float4 v4 = *reinterpret_cast<const float4*>(sc + TN + c0 + 2 * e);
                                y = mul2(y, make_float2(v4.x, v4.y));
                                z = mul2(z, make_float2(v4.z, v4.w));
                                if (masked) {  // nothing from a token that the row does not see, whatever its scale
                                    if (!((bits >> (2 * e)) & 1)) y.x = 0.f;
                                    if (!((bits >> (2 * e + 1)) & 1)) y.y = 0.f;
                                    if (!((bits >> (2 * e + 2)) & 1)) z.x = 0.f;
                                    if (!((bits >> (2 * e + 3)) & 1)) z.y = 0.f;
                                }
                            }
                            p[e] = E4M3 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
                            p[e + 1] = E4M3 ? pack_f16(z.x, z.y) : pack_bf16(z.x, z.y);
                        }
                        tmem_st16(s0 + (half * HC + c0) / 2, p);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.pfull[b]);
                if (!busy && !ok) break;
            }
            // ---- the segment's output
            ok = ok && all_wait(&B.odone, (i - 1) & 1, abort_flag, wlim);
            if (busy ? pair_any(pair, !ok) : !ok) { ok = false; break; }
            tc_fence_after();
            const bool odd = !E4M3 && *reinterpret_cast<volatile int*>(&B.odd) != 0;
            if (busy) {
                row_top[half * 128 + m] = l2.x + l2.y;
                pair_sync(pair);
                const float l = row_top[m] + row_top[128 + m];
                const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
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
                    tmem_ld32(tmem + lane_off + c0, o);
                    tmem_wait_ld();
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
                pair_sync(pair);  // the sums are read
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

// The cache's rows [n_pages * Hk * page, D] bf16; boxes of 64 elements x the
// rows of a page that one tile can take, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* ptr, const CacheView& c, int rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)c.D, (cuuint64_t)((c.n_pages * c.Hk) << c.page_shift)};
    cuuint64_t strides[1] = {(cuuint64_t)c.D * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3>
cudaError_t launch_tc(const TreeArgs& a, cudaStream_t s) {
    using C = Tc<D, E4M3>;
    CUtensorMap mk = {}, mv = {};
    const int page = 1 << a.c.page_shift, run = page < C::TN ? page : C::TN;
    if (!E4M3 && (!make_map(&mk, a.c.k, a.c, run) || !make_map(&mv, a.c.v, a.c, run))) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D, E4M3><<<a.grid, kTcThreads, C::kSmem, s>>>(a, mk, mv);
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
