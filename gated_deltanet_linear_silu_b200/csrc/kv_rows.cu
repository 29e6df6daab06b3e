// Rows of the softmax-attention layer ("7.6 Qwen3.5: linear-attention hybrid",
// config table and attention layers: RMSNorm of each query and key head, a
// quarter of each head rotated by position): the norm and the rotation, the
// writes to the paged cache and the reads from it.
//
//   y = x / sqrt(mean(x^2) + eps) * w                 per (token, head)
//   (a, b) -> (a cos - b sin, b cos + a sin)          pairs of the first `rotary`
//                                                     elements, angle pos * inv_freq
//   e4m3 row: scale = amax / 448, code = x / scale    nearest even
//
// All of it is HBM-bound (each element read once, written once) if few
// instructions go with a 16-byte piece. A warp takes one token (or a share of
// its heads, where tokens are few) and walks its heads, 32 / LPR rows at a time,
// LPR lanes of sixteen elements to a row: the norm and amax are shuffles within
// the lane group, and the token's place in the cache and its angles are looked
// up once for all its heads. Where pairs are the two halves of the rotated part,
// a lane of that part takes eight elements of either half, so that a pair stays
// in one lane and the rotation exchanges nothing.
//
// Measured: norm and rotation of 16384 tokens, 8 + 2 heads of 256, bf16: 39 us
// (168 MB, 4.4 TB/s); 32771 tokens of 8 heads of 128 into an e4m3 cache: 45 us
// (203 MB, 4.5 TB/s); 131101 such tokens read back: 153 us (814 MB, 5.3 TB/s, 81 %
// of a copy's rate). The first two reach neither limit (61 and 68 % of the issue slots):
// a warp asks for a token's rows when the one before is stored, and waits for them. With
// eight elements a lane, and more instructions, they took 46 and 62 us.
//
// The angle's turns, pos * inv_freq / (2 pi), are taken in fp64 and reduced to
// [-1/2, 1/2] there: in fp32 a position of 2^18 would lose 2^-6 of a radian.
#include <cfloat>

#include "kv_page.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 2;  // row groups of a warp in flight

// Eight consecutive elements, as loaded.
template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
__device__ __forceinline__ void put8(uint16_t* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// x / s rounded once, given r close to 1 / s (Markstein's correction: the
// remainder of x r, times r, added to it). Where the quotient is a number of the
// format -- the ties of the rounding that follows among them -- it comes out
// exactly. No step may leave the normal range.
__device__ __forceinline__ float corrected(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}
__device__ __forceinline__ float reciprocal(float s) {  // within an ulp, for normal s: one Newton step
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

__device__ __forceinline__ float max_abs_nan(float m, float x) {  // max(m, |x|), NaN if either is
    float y;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(y) : "f"(m), "f"(x));
    return y;
}

// Stores one row's sixteen elements per lane in the cache, eight at p0 and eight
// at p1; every lane of the group takes part (the amax is the group's). A row
// with an element that is not finite is stored as scale NaN: it reads back as
// NaN.
template <int LPR>
__device__ __forceinline__ void put_cache(int e4m3, uint8_t* row, float* scale_at, int l, int p0, int p1, bool on,
                                          float (&x)[16]) {
    if (!e4m3) {
        if (on) {
            put8(reinterpret_cast<uint16_t*>(row) + p0, x);
            put8(reinterpret_cast<uint16_t*>(row) + p1, x + 8);
        }
        return;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max_abs_nan(m, x[i]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale;
    if (m >= 0x1p-100f && m <= 0x1p100f) {
        scale = corrected(m, 448.f, 1.f / 448.f);
        const float r = reciprocal(scale);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = corrected(x[i], scale, r);
    } else {
        const bool finite = m <= FLT_MAX;
        scale = finite ? m / 448.f : __uint_as_float(0x7FC00000u);
        const bool zero = !finite || scale == 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = zero ? 0.f : __fdiv_rn(x[i], scale);
    }
    if (!on) return;
    *reinterpret_cast<uint2*>(row + p0) = to_e4m3x8(x);
    *reinterpret_cast<uint2*>(row + p1) = to_e4m3x8(x + 8);
    if (l == 0) *scale_at = scale;
}

// Groups of 32 / LPR rows of a token: queries, keys, values. 1 << share_shift
// warps take a token's groups in turn; INTER: pairs are neighbours.
template <typename T, int LPR, int MODE, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? (MODE == kCacheWrite ? 4 : 3) : 2)
rows_kernel(RowsArgs a, int share_shift) {
    extern __shared__ __align__(16) float trig[];  // per warp: cos [half], sin [half]
    // sequences that reach past the last packed row: written up to there
    if (MODE != kNormRope && blockIdx.x == 0 && threadIdx.x == 0 && a.p.cu[a.p.N] > a.T) set_status(a.status, kStatusBadSeqlens);
    constexpr int RW = 32 / LPR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPR, sub = lane / LPR;
    const int D = a.D, half = a.rotary >> 1;
    const bool on = 16 * l < D;
    const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
    const int part = (int)(gw & ((1 << share_shift) - 1));
    const int nq = MODE == kCacheWrite ? 0 : (a.H + RW - 1) / RW, nk = (a.Hk + RW - 1) / RW;
    const int groups = nq + (MODE == kNormRope ? nk : 2 * nk);
    // This lane's elements: eight of either half of the row, or, where pairs are the
    // halves of a rotated part, of either half of that part or of the rest.
    const bool turned = MODE != kCacheWrite && !INTER && 16 * l < a.rotary;
    const int v0 = 8 * l, v1 = (D >> 1) + 8 * l;
    const int p0 = MODE == kCacheWrite || INTER || turned ? v0 : half + v0;
    const int p1 = MODE == kCacheWrite || INTER ? v1 : turned ? half + v0 : v1;
    const float inv_d = 1.f / (float)D;
    float* const cw = trig + warp * 2 * half;
    const int64_t stride = ((int64_t)gridDim.x * kWarps) >> share_shift;
    for (int64_t t = gw >> share_shift; t < a.T; t += stride) {
        const T* q0 = static_cast<const T*>(a.q) + t * a.ld_q + sub * D;
        const T* k0 = static_cast<const T*>(a.k) + t * a.ld_k + sub * D;
        const T* vt = static_cast<const T*>(a.v) + t * a.ld_v + sub * D;
        Vec8<T> raw[kBatch][2] = {};  // (lanes past the row keep zeros)
        auto load = [&](int g0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int g = g0 + (u << share_shift);
                if (g >= groups) break;
                if (MODE != kCacheWrite && g < nq) {
                    if (on && g * RW + sub < a.H) {
                        raw[u][0].load(q0 + g * (RW * D) + p0);
                        raw[u][1].load(q0 + g * (RW * D) + p1);
                    }
                } else if (g < nq + nk) {
                    if (on && (g - nq) * RW + sub < a.Hk) {
                        raw[u][0].load(k0 + (g - nq) * (RW * D) + p0);
                        raw[u][1].load(k0 + (g - nq) * (RW * D) + p1);
                    }
                } else if (MODE != kNormRope) {
                    if (on && (g - nq - nk) * RW + sub < a.Hk) {
                        raw[u][0].load(vt + (g - nq - nk) * (RW * D) + v0);
                        raw[u][1].load(vt + (g - nq - nk) * (RW * D) + v1);
                    }
                }
            }
        };
        load(part);
        if (MODE != kCacheWrite) {
            const double pos = (double)a.pos[t] * 0.15915494309189533577;  // 1 / (2 pi)
            __syncwarp();  // the last token's angles are read
            for (int i = lane; i < half; i += 32) {
                const double turns = pos * a.inv_freq[i];
                sincospif(2.f * (float)(turns - rint(turns)), &cw[half + i], &cw[i]);
            }
            __syncwarp();
        }
        int64_t where = 0;
        if (MODE != kNormRope) {
            where = token_row(a.p, a.c, t);
            if (where < 0) {
                if (where == kRowBad && lane == 0) set_status(a.status, kStatusBadSeqlens);
                continue;
            }
            where += (int64_t)sub << a.c.page_shift;
        }
        // this lane group's first cached row of the token; RW heads further is `step` rows on
        const int row_bytes = a.c.e4m3 ? D : 2 * D, step = RW << a.c.page_shift;
        uint8_t* const kd = static_cast<uint8_t*>(a.c.k) + where * row_bytes;
        uint8_t* const vd = static_cast<uint8_t*>(a.c.v) + where * row_bytes;
        float* const ks = a.c.k_scale + where;
        float* const vs = a.c.v_scale + where;
        T* const qo = static_cast<T*>(a.q_out) + t * a.H * D + sub * D;
        T* const ko = static_cast<T*>(a.k_out) + t * a.Hk * D + sub * D;
        float w[16];            // weights of the rows at hand
        const float* held = nullptr;
        auto normed = [&](float (&x)[16], const float* weights) {
            if (held != weights) {  // (uniform: queries come first, then keys)
                held = weights;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 y = on ? __ldg(reinterpret_cast<const float4*>(weights + (e < 8 ? p0 + e : p1 + e - 8)))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                    w[e] = y.x; w[e + 1] = y.y; w[e + 2] = y.z; w[e + 3] = y.w;
                }
            }
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * w[e];
            auto turn = [](float& p, float& q, float c, float s) {
                const float y = p * c - q * s;
                q = q * c + p * s;
                p = y;
            };
            if (INTER) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = h ? p1 : p0;
                    if (at >= a.rotary) continue;
                    const float4 c4 = *reinterpret_cast<const float4*>(cw + (at >> 1));
                    const float4 s4 = *reinterpret_cast<const float4*>(cw + half + (at >> 1));
                    turn(x[8 * h], x[8 * h + 1], c4.x, s4.x);
                    turn(x[8 * h + 2], x[8 * h + 3], c4.y, s4.y);
                    turn(x[8 * h + 4], x[8 * h + 5], c4.z, s4.z);
                    turn(x[8 * h + 6], x[8 * h + 7], c4.w, s4.w);
                }
            } else if (turned) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 c4 = *reinterpret_cast<const float4*>(cw + p0 + e);
                    const float4 s4 = *reinterpret_cast<const float4*>(cw + half + p0 + e);
                    turn(x[e], x[e + 8], c4.x, s4.x);
                    turn(x[e + 1], x[e + 9], c4.y, s4.y);
                    turn(x[e + 2], x[e + 10], c4.z, s4.z);
                    turn(x[e + 3], x[e + 11], c4.w, s4.w);
                }
            }
        };
        for (int g0 = part; g0 < groups; g0 += kBatch << share_shift) {
            if (g0 != part) load(g0);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int g = g0 + (u << share_shift);
                if (g >= groups) break;
                float x[16];
                raw[u][0].get(x);
                raw[u][1].get(x + 8);
                if (MODE != kCacheWrite && g < nq) {
                    normed(x, a.q_w);
                    if (on && g * RW + sub < a.H) {
                        put8(qo + g * (RW * D) + p0, x);
                        put8(qo + g * (RW * D) + p1, x + 8);
                    }
                } else if (g < nq + nk) {
                    if (MODE != kCacheWrite) normed(x, a.k_w);
                    const bool live = on && (g - nq) * RW + sub < a.Hk;
                    if (MODE == kNormRope) {
                        if (live) {
                            put8(ko + (g - nq) * (RW * D) + p0, x);
                            put8(ko + (g - nq) * (RW * D) + p1, x + 8);
                        }
                    } else {
                        const int at = (g - nq) * step;
                        put_cache<LPR>(a.c.e4m3, kd + (int64_t)at * row_bytes, ks + at, l, p0, p1, live, x);
                    }
                } else if (MODE != kNormRope) {
                    const int at = (g - nq - nk) * step;
                    put_cache<LPR>(a.c.e4m3, vd + (int64_t)at * row_bytes, vs + at, l, v0, v1,
                                   on && (g - nq - nk) * RW + sub < a.Hk, x);
                }
            }
        }
    }
}

// Warps to a token (log2): more while the GPU would not be full without them.
int share_of_token(int64_t T, int groups) {
    int s = 0;
    while (s < 3 && (T << s) < 2 * kWarps * (int64_t)sm_count() && (2 << s) <= groups) ++s;
    return s;
}

// CTAs for that many warps: at most eight to an SM, which then walk the tokens.
unsigned grid_of(int64_t warps) {
    const int64_t need = (warps + kWarps - 1) / kWarps, most = 8 * (int64_t)sm_count();
    return (unsigned)(need < most ? need : most);
}

template <typename T, int LPR>
cudaError_t launch_lpr(const RowsArgs& a, RowsMode mode, cudaStream_t s) {
    constexpr int RW = 32 / LPR;
    const int nk = (a.Hk + RW - 1) / RW;
    const int groups = mode == kCacheWrite ? 2 * nk : (a.H + RW - 1) / RW + (mode == kNormRope ? nk : 2 * nk);
    const int share = share_of_token(a.T, groups);
    const unsigned grid = grid_of(a.T << share);
    const size_t smem = mode == kCacheWrite ? 0 : sizeof(float) * kWarps * a.rotary;
    switch (mode) {
        case kNormRope:
            if (a.interleaved) rows_kernel<T, LPR, kNormRope, true><<<grid, kThreads, smem, s>>>(a, share);
            else rows_kernel<T, LPR, kNormRope, false><<<grid, kThreads, smem, s>>>(a, share);
            break;
        case kNormRopeCache:
            if (a.interleaved) rows_kernel<T, LPR, kNormRopeCache, true><<<grid, kThreads, smem, s>>>(a, share);
            else rows_kernel<T, LPR, kNormRopeCache, false><<<grid, kThreads, smem, s>>>(a, share);
            break;
        case kCacheWrite: rows_kernel<T, LPR, kCacheWrite, false><<<grid, kThreads, smem, s>>>(a, share); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RowsArgs& a, RowsMode mode, cudaStream_t s) {
    if (a.D <= 32) return launch_lpr<T, 2>(a, mode, s);
    if (a.D <= 64) return launch_lpr<T, 4>(a, mode, s);
    if (a.D <= 128) return launch_lpr<T, 8>(a, mode, s);
    return launch_lpr<T, 16>(a, mode, s);
}

// ---- reading back, the same walk: key rows, then value rows of a token.
template <typename T, int LPR, bool E4M3>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a, int share_shift) {
    constexpr int RW = 32 / LPR, kAhead = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPR, sub = lane / LPR;
    const int D = a.c.D, Hk = a.c.Hk;
    const bool on = 8 * l < D;
    const int64_t gw = (int64_t)blockIdx.x * kWarps + warp, t = gw >> share_shift;
    const int part = (int)(gw & ((1 << share_shift) - 1));
    if (t >= a.T) return;
    const int64_t where = token_row(a.p, a.c, t);
    if (where < 0) {
        if (where == kRowBad && lane == 0) set_status(a.status, kStatusBadSeqlens);
        return;
    }
    const int nk = (Hk + RW - 1) / RW;
    for (int g0 = part; g0 < 2 * nk; g0 += kAhead << share_shift) {
        uint4 raw[kAhead];
        float sc[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = g0 + (u << share_shift);
            if (g >= 2 * nk) break;
            const int j = (g < nk ? g : g - nk) * RW + sub;
            if (!on || j >= Hk) continue;
            const int64_t row = where + ((int64_t)j << a.c.page_shift);
            const uint8_t* src = static_cast<const uint8_t*>(g < nk ? a.c.k : a.c.v);
            if (E4M3) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src + row * D + 8 * l));
                raw[u] = make_uint4(w.x, w.y, 0, 0);
                sc[u] = __ldg((g < nk ? a.c.k_scale : a.c.v_scale) + row);
            } else {
                raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + 2 * (row * D + 8 * l)));
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = g0 + (u << share_shift);
            if (g >= 2 * nk) break;
            const int j = (g < nk ? g : g - nk) * RW + sub;
            if (!on || j >= Hk) continue;
            T* dst = static_cast<T*>(g < nk ? a.k : a.v) + (t * Hk + j) * D;
            float f[8];
            if (E4M3) {
                from_e4m3x8(make_uint2(raw[u].x, raw[u].y), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= sc[u];
            } else if (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(dst + 8 * l) = raw[u];
                continue;
            } else {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(w[e] << 16);
                    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
                }
            }
            put8(dst + 8 * l, f);
        }
    }
}

template <typename T, int LPR>
cudaError_t launch_read(const ReadArgs& a, cudaStream_t s) {
    constexpr int RW = 32 / LPR;
    const int share = share_of_token(a.T, 2 * ((a.c.Hk + RW - 1) / RW));
    const unsigned grid = (unsigned)(((a.T << share) + kWarps - 1) / kWarps);
    if (a.c.e4m3) read_kernel<T, LPR, true><<<grid, kThreads, 0, s>>>(a, share);
    else read_kernel<T, LPR, false><<<grid, kThreads, 0, s>>>(a, share);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_read_type(const ReadArgs& a, cudaStream_t s) {
    if (a.c.D <= 16) return launch_read<T, 2>(a, s);
    if (a.c.D <= 32) return launch_read<T, 4>(a, s);
    if (a.c.D <= 64) return launch_read<T, 8>(a, s);
    if (a.c.D <= 128) return launch_read<T, 16>(a, s);
    return launch_read<T, 32>(a, s);
}

// ---- accepting a path: one CTA per sequence. Row base + a takes row base +
// path[a]; the path increases, so no source is overwritten before its turn. A
// thread owns one 16-byte column (or the scale) of a head through the whole
// path, eight rows loaded before they are stored.
template <typename V>
__device__ __forceinline__ void move_column(V* data, int64_t stride, const int64_t* src, const int64_t* dst, int count) {
    constexpr int kAhead = 8;
    for (int a0 = 0; a0 < count; a0 += kAhead) {
        V x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (a0 + u < count) x[u] = data[src[a0 + u] * stride];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (a0 + u < count) data[dst[a0 + u] * stride] = x[u];
    }
}

__global__ void __launch_bounds__(kThreads) accept_kernel(AcceptArgs a) {
    __shared__ int64_t src[kMaxNodes], dst[kMaxNodes];
    __shared__ int bad;
    const int n = blockIdx.x, tid = threadIdx.x;
    const int64_t first = a.p.cu[n], last = a.p.cu[n + 1];
    const int64_t nodes = last - first, base = (int64_t)a.p.lens[n] - nodes;
    const int32_t* path = a.path + (int64_t)n * a.M;
    if (tid == 0) bad = nodes < 0 || base < 0;
    __syncthreads();
    int at = -1;
    if (tid < a.M) {
        at = path[tid];
        if (at >= 0) {
            // increasing, without a gap, inside the draft
            if (at >= nodes || (tid > 0 && (path[tid - 1] < 0 || path[tid - 1] >= at))) bad = 1;
            src[tid] = page_row(a.p, a.c, n, base + at);
            dst[tid] = page_row(a.p, a.c, n, base + tid);
            if (src[tid] < 0 || dst[tid] < 0) bad = 1;
        }
    }
    const int count = __syncthreads_count(at >= 0);
    if (bad) {
        if (tid == 0) {
            set_status(a.status, kStatusBadSeqlens);
            a.new_lens[n] = a.p.lens[n];
        }
        return;
    }
    if (tid == 0) a.new_lens[n] = (int32_t)(base + count);
    // the leading nodes that already stand where they belong are not moved
    int skip = 0;
    while (skip < count && src[skip] == dst[skip]) ++skip;
    if (skip == count) return;
    const int cols = a.c.D * (a.c.e4m3 ? 1 : 2) / 16;
    const int per = cols + (a.c.e4m3 ? 1 : 0);
    for (int x = tid; x < 2 * a.c.Hk * per; x += kThreads) {
        const int col = x % per, hk = (x / per) % a.c.Hk;
        const bool is_v = x / per >= a.c.Hk;
        const int64_t head = (int64_t)hk << a.c.page_shift;
        if (col < cols)
            move_column(static_cast<uint4*>(is_v ? a.c.v : a.c.k) + head * cols + col, cols, src + skip, dst + skip,
                        count - skip);
        else
            move_column((is_v ? a.c.v_scale : a.c.k_scale) + head, 1, src + skip, dst + skip, count - skip);
    }
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, RowsMode mode, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    return a.is_bf16 ? launch_type<uint16_t>(a, mode, s) : launch_type<float>(a, mode, s);
}

cudaError_t launch_kv_read(const ReadArgs& a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    return a.out_bf16 ? launch_read_type<uint16_t>(a, s) : launch_read_type<float>(a, s);
}

cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s) {
    accept_kernel<<<(unsigned)a.p.N, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
