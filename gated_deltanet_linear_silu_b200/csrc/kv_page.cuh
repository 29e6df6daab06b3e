// Device helpers of the paged key/value cache.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace gdn {

// Cache row of head 0 at position `pos` of sequence n (add hk << page_shift for
// head hk; times D for the element); -1 where the page table has no such page.
__device__ __forceinline__ int64_t page_row(const PageArgs& p, const CacheView& c, int n, int64_t pos) {
    const int64_t slot = pos >> c.page_shift;
    if (pos < 0 || slot >= p.max_pages) return -1;
    const int id = __ldg(p.table + (int64_t)n * p.max_pages + slot);
    if (id < 0 || id >= c.n_pages) return -1;
    return (((int64_t)id * c.Hk) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

constexpr int64_t kRowNone = -1;  // a row behind the last sequence
constexpr int64_t kRowBad = -2;   // bounds or page that the arguments do not allow

// Cache row of packed token t.
__device__ __forceinline__ int64_t token_row(const PageArgs& p, const CacheView& c, int64_t t) {
    if (t >= p.cu[p.N]) return kRowNone;
    const int n = find_sequence(p.cu, p.N, t);
    const int64_t a = p.cu[n], b = p.cu[n + 1];
    if (t < a || t >= b) return kRowBad;
    const int64_t row = page_row(p, c, n, (int64_t)p.lens[n] - b + t);
    return row < 0 ? kRowBad : row;
}

// Eight e4m3 values from fp32, to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint2 to_e4m3x8(const float* x) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        h[i] = r;
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Eight fp32 values from e4m3 (exact).
__device__ __forceinline__ void from_e4m3x8(uint2 u, float (&x)[8]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        uint32_t f;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(f));
    }
}

}  // namespace gdn
