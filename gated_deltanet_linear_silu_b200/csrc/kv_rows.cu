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
// All of it is HBM-bound (each element read once, written once); a row is held
// by a group of D / 8 lanes, eight elements each, so that a bf16 row moves in
// 16-byte vectors and the norm and amax are shuffles within the group. The
// sine and cosine of a token serve all its heads: a CTA takes whole tokens and
// computes them once into shared memory. The angle's turns, pos * inv_freq /
// (2 pi), are taken in fp64 and reduced to [-1/2, 1/2] there: in fp32 a
// position of 2^18 would lose 2^-6 of a radian.
#include <cfloat>

#include "kv_page.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 4;  // rows of a lane group in flight
constexpr int kMaxTokens = 8;  // tokens of a CTA

template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
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
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
__device__ __forceinline__ void put8(uint16_t* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Stores one row's eight elements per lane in the cache; every lane of the
// group takes part (the amax is the group's). A row with an element that is
// not finite is stored as scale NaN: it reads back as NaN.
template <int LPR>
__device__ __forceinline__ void put_cache(const CacheView& c, bool is_v, int64_t row, int l, bool on, float (&x)[8]) {
    if (!c.e4m3) {
        if (on) put8(static_cast<uint16_t*>(is_v ? c.v : c.k) + row * c.D + 8 * l, x);
        return;
    }
    uint32_t m = 0;  // bits of |x| order as the values do, with inf and NaN on top
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < 0x7F800000u;
    const float scale = finite ? __uint_as_float(m) / 448.f : __uint_as_float(0x7FC00000u);
    const bool zero = !finite || scale == 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = zero ? 0.f : x[i] / scale;
    if (!on) return;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + row * c.D + 8 * l) = to_e4m3x8(x);
    if (l == 0) (is_v ? c.v_scale : c.k_scale)[row] = scale;
}

// One CTA: tb tokens, all their rows (q then k then v heads of each token).
template <typename T, int LPR, int MODE>
__global__ void __launch_bounds__(kThreads) rows_kernel(RowsArgs a, int tb) {
    extern __shared__ float trig[];  // cos [tb][half], then sin [tb][half]
    __shared__ int64_t where[kMaxTokens];
    constexpr int RW = 32 / LPR;  // rows of a warp's pass
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int l = lane % LPR, sub = lane / LPR;
    const int D = a.D, half = a.rotary >> 1;
    const bool on = 8 * l < D;
    const int H = MODE == kCacheWrite ? 0 : a.H;
    const int R = H + (MODE == kNormRope ? a.Hk : 2 * a.Hk);
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int nt = (int)(a.T - t0 < tb ? a.T - t0 : tb);
    const int rows = nt * R;
    constexpr int kStep = kWarps * RW;

    // Token and head slot of row r, and its load.
    Vec8<T> raw[kBatch];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int r = r0 + u * kStep + warp * RW + sub;
            if (r >= rows || !on) continue;
            const int64_t t = t0 + r / R;
            const int j = r % R;
            const T* src = j < H ? static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)j * D
                         : j < H + a.Hk ? static_cast<const T*>(a.k) + t * a.ld_k + (int64_t)(j - H) * D
                                        : static_cast<const T*>(a.v) + t * a.ld_v + (int64_t)(j - H - a.Hk) * D;
            raw[u].load(src + 8 * l);
        }
    };
    load(0);
    if (MODE != kNormRope && tid < nt) {
        const int64_t row = token_row(a.p, a.c, t0 + tid);
        where[tid] = row;
        if (row == kRowBad) set_status(a.status, kStatusBadSeqlens);
    }
    float wq[8], wk[8];
    if (MODE != kCacheWrite) {
        for (int i = tid; i < nt * half; i += kThreads) {
            const double turns = (double)a.pos[t0 + i / half] * a.inv_freq[i % half] * 0.15915494309189533577;
            float s, c;
            sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
            trig[i] = c;
            trig[tb * half + i] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wq[i] = on ? a.q_w[8 * l + i] : 0.f;
            wk[i] = on ? a.k_w[8 * l + i] : 0.f;
        }
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kBatch * kStep) {
        if (r0 > 0) load(r0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int rw = r0 + u * kStep + warp * RW;  // first row of the warp's pass
            if (rw >= rows) break;
            const int r = rw + sub;
            const bool live = r < rows;
            const int i = live ? r / R : 0, j = live ? r % R : 0;
            float x[8];
            if (live && on) raw[u].get(x);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            if (MODE != kCacheWrite) {
                const bool normed = j < H + a.Hk;
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e] * inv * (j < H ? wq[e] : wk[e]);
                const int c0 = 8 * l;
                const bool turned = c0 < a.rotary;
                const float* cs = trig + i * half;
                const float* sn = cs + tb * half;
                if (a.interleaved) {
                    if (turned) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float c = cs[(c0 + e) >> 1], s = sn[(c0 + e) >> 1];
                            const float p = y[e], q = y[e + 1];
                            y[e] = p * c - q * s;
                            y[e + 1] = q * c + p * s;
                        }
                    }
                } else {
                    // the pair's other element sits half / 8 lanes away (rotary is a multiple of 16)
                    const bool first = c0 < half;
                    const int peer = turned ? (first ? lane + half / 8 : lane - half / 8) : lane;
                    const int at = turned ? (first ? c0 : c0 - half) : 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p = __shfl_sync(0xffffffffu, y[e], peer);
                        if (turned) y[e] = y[e] * cs[at + e] + (first ? -p : p) * sn[at + e];
                    }
                }
                if (normed) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = y[e];
                }
            }
            if (MODE == kNormRope) {
                if (live && on) {
                    const int64_t t = t0 + i;
                    T* dst = j < H ? static_cast<T*>(a.q_out) + (t * H + j) * D
                                   : static_cast<T*>(a.k_out) + (t * a.Hk + j - H) * D;
                    put8(dst + 8 * l, x);
                }
            } else {
                const int64_t row = live ? where[i] : kRowNone;
                const bool store = row >= 0 && on;
                if (MODE == kNormRopeCache && j < H && store)
                    put8(static_cast<T*>(a.q_out) + ((t0 + i) * H + j) * D + 8 * l, x);
                const int hk = j - H;
                if (!__any_sync(0xffffffffu, hk >= 0)) continue;  // queries only
                const bool is_v = hk >= a.Hk;
                put_cache<LPR>(a.c, is_v, row + ((int64_t)(is_v ? hk - a.Hk : hk) << a.c.page_shift), l,
                               store && hk >= 0, x);
            }
        }
    }
}

template <typename T, int LPR>
cudaError_t launch_lpr(const RowsArgs& a, RowsMode mode, cudaStream_t s) {
    // whole tokens per CTA: as many (up to 8) as still leave two CTAs for every SM
    int tb = kMaxTokens;
    while (tb > 1 && (a.T + tb - 1) / tb < 2 * sm_count()) tb >>= 1;
    const unsigned grid = (unsigned)((a.T + tb - 1) / tb);
    const size_t smem = mode == kCacheWrite ? 0 : sizeof(float) * tb * a.rotary;
    switch (mode) {
        case kNormRope: rows_kernel<T, LPR, kNormRope><<<grid, kThreads, smem, s>>>(a, tb); break;
        case kNormRopeCache: rows_kernel<T, LPR, kNormRopeCache><<<grid, kThreads, smem, s>>>(a, tb); break;
        case kCacheWrite: rows_kernel<T, LPR, kCacheWrite><<<grid, kThreads, smem, s>>>(a, tb); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RowsArgs& a, RowsMode mode, cudaStream_t s) {
    if (a.D <= 16) return launch_lpr<T, 2>(a, mode, s);
    if (a.D <= 32) return launch_lpr<T, 4>(a, mode, s);
    if (a.D <= 64) return launch_lpr<T, 8>(a, mode, s);
    if (a.D <= 128) return launch_lpr<T, 16>(a, mode, s);
    return launch_lpr<T, 32>(a, mode, s);
}

// ---- reading back: a CTA takes 16 tokens (one page's run, where pages are that
// long), a lane eight elements of a row.
constexpr int kReadTokens = 16;

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a) {
    __shared__ int64_t where[kReadTokens];
    const int tid = threadIdx.x, D = a.c.D, Hk = a.c.Hk, cols = D >> 3;
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    const int nt = (int)(a.T - t0 < kReadTokens ? a.T - t0 : kReadTokens);
    if (tid < nt) {
        const int64_t row = token_row(a.p, a.c, t0 + tid);
        where[tid] = row;
        if (row == kRowBad) set_status(a.status, kStatusBadSeqlens);
    }
    __syncthreads();
    const bool is_v = blockIdx.y != 0;
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.c.v : a.c.k);
    const float* scales = is_v ? a.c.v_scale : a.c.k_scale;
    T* dst = static_cast<T*>(is_v ? a.v : a.k) + t0 * Hk * D;
    const int items = nt * Hk * cols;
    for (int x0 = tid; x0 < items; x0 += kBatch * kThreads) {
        uint4 raw[kBatch];
        float sc[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int x = x0 + u * kThreads;
            if (x >= items) break;
            const int r = x / cols, e = 8 * (x - r * cols), i = r / Hk;
            if (where[i] < 0) continue;
            const int64_t row = where[i] + ((int64_t)(r - i * Hk) << a.c.page_shift);
            if (E4M3) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src + row * D + e));
                raw[u] = make_uint4(w.x, w.y, 0, 0);
                sc[u] = scales[row];
            } else {
                raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + 2 * (row * D + e)));
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int x = x0 + u * kThreads;
            if (x >= items) break;
            if (where[x / cols / Hk] < 0) continue;
            float f[8];
            if (E4M3) {
                from_e4m3x8(make_uint2(raw[u].x, raw[u].y), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= sc[u];
            } else {
                Vec8<uint16_t> b;
                b.u = raw[u];
                b.get(f);
            }
            put8(dst + 8 * (int64_t)x, f);
        }
    }
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
    const dim3 grid((unsigned)((a.T + kReadTokens - 1) / kReadTokens), 2);
    if (a.out_bf16) {
        if (a.c.e4m3) read_kernel<uint16_t, true><<<grid, kThreads, 0, s>>>(a);
        else read_kernel<uint16_t, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.c.e4m3) read_kernel<float, true><<<grid, kThreads, 0, s>>>(a);
        else read_kernel<float, false><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s) {
    accept_kernel<<<(unsigned)a.p.N, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
