// Shared device code of the tree-attention kernels: the line of work, its
// shares and segments, the workspace, and small helpers.
//
// Query rows of a (sequence, key/value head) -- (node, query head of the group)
// pairs, node-major -- are cut into row tiles. The line of a row tile rt is the
// token tiles of all (sequence, head) units that have it, sequences in order.
// The grid is dealt to the row tiles in proportion to their lines, and each
// CTA takes an equal stretch of its row tile's line; CTAs of different row
// tiles with equal lines walk the same cache rows at the same time, so that
// all but the first read them from L2. A stretch is walked in segments, one per
// unit it touches. A unit within one CTA is finished there; one that spans CTAs
// leaves a partial (m, l, o unnormalised) in each, which join_kernel adds up in
// the CTAs' order: the result does not depend on timing.
#pragma once

#include "kv_page.cuh"

namespace gdn {

constexpr int kTcRows = 128;    // query rows of a row tile (tcgen05 kernel)
constexpr int kTcTile = 64;     // tokens of its tiles
constexpr int kMaxRowTiles = 32;
template <bool B>
struct Bool {
    static constexpr bool value = B;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;  // growth of a row's largest weight (log2) that moves its reference
// Where a move puts the largest weight (log2). f16 numerators (e4m3 caches) stand as
// high as the growth and the type's 2^16 allow: they keep eleven bits down to 2^-21 of
// the largest, and what is below is off by 2^-32 of it at most, so that 2^17 tokens of
// such weights together move a sum by 2^-15 of its largest term.
template <bool E4M3>
constexpr float kLift = E4M3 ? 7.f : 0.f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// f16x2 of the two e4m3 codes in the low half of x (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(x));
    return y;
}

// The power of two that takes a row of bf16 queries to f16, and back: it puts the
// largest magnitude, whose bits are `top`, in [2^14, 2^15). The least that f16 keeps is
// 2^-24, so that an element's eight bits are exact down to 2^-31 of the largest, and
// what is below is off by 2^-39 of it at most: less than the fp32 sums of the scores.
// Rows below 2^-112 stay lower; the finite elements of one that is not finite fit.
__device__ __forceinline__ void query_scale(uint32_t top, float& down, float& up) {
    uint32_t e = top >> 7;  // 127 + exponent
    e = e < 15u ? 15u : e > 254u ? 254u : e;
    down = __uint_as_float((268u - e) << 23);
    up = __uint_as_float((e - 14u) << 23);
}

// log2 of a value row's scale for the running reference: at least -92, so that a
// weight without its scale, up to 2^(92 + kLift + kLazy), and 2^20 of them stay in
// fp32's range.
__device__ __forceinline__ float log2_scale(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return fmaxf(y, -92.f);
}

// Zeroes the halves of a bf16 pair that are not finite; true if there was one.
__device__ __forceinline__ bool zero_non_finite(uint32_t& x) {
    const uint32_t y = x;
    if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
    if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
    return x != y;
}

// Asynchronous copies that write zeros where `on` is false (nothing is read).
__device__ __forceinline__ void cp_async_zfill16(void* dst, const void* src, bool on) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_zfill4(void* dst, const void* src, bool on) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int n = on ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Positions are counted in 32 bits, a few tiles past a sequence's end as well.
constexpr int kMaxLen = 0x7FFFFFFF - 1023;

// Sequence n's draft and length, checked; no nodes where there is nothing to do.
struct Seq {
    int first, nodes, len;  // first packed token, drafted tokens, cached tokens
    bool bad;
};
__device__ __forceinline__ Seq load_seq(const TreeArgs& a, int n) {
    Seq q;
    q.first = a.p.cu[n];
    const int64_t end = a.p.cu[n + 1], nodes = end - q.first;
    q.len = a.p.lens[n];
    q.bad = q.first < 0 || nodes < 0 || end > a.T || nodes > a.max_nodes || q.len < nodes ||
            q.len > ((int64_t)a.p.max_pages << a.c.page_shift) || q.len > kMaxLen;
    q.nodes = q.bad ? 0 : (int)nodes;
    return q;
}

// Workspace: for every unit ([row_tiles][N * Hk]) where its partials are; per
// CTA two partials (of the segment at the start of its stretch, and of one that
// starts later), each m, l [slot_rows] and o [slot_rows][D].
struct UnitParts {
    int first;  // partial of the unit's first segment: 2 CTA + (0 or 1)
    int last;   // CTA of its last one; the CTAs between have theirs at 2 CTA
};
__host__ __device__ inline size_t units_bytes(int row_tiles, int N, int Hk) {
    return (sizeof(UnitParts) * row_tiles * N * Hk + 255) / 256 * 256;
}
__host__ __device__ inline size_t slot_floats(int D, int slot_rows) { return (size_t)slot_rows * (D + 2); }

__device__ __forceinline__ UnitParts* unit_parts(const TreeArgs& a, int rt, int n, int hk) {
    return static_cast<UnitParts*>(a.workspace) + ((int64_t)rt * a.p.N + n) * a.c.Hk + hk;
}
__device__ __forceinline__ float* partial_base(const TreeArgs& a) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + units_bytes(a.row_tiles, a.p.N, a.c.Hk));
}

// a / b of non-negative numbers: 64-bit division is a long call, and these
// mostly fit 32.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int ROWS>
__device__ __forceinline__ int seq_row_tiles(const TreeArgs& a, const Seq& q) {
    return (q.nodes * (a.H / a.c.Hk) + ROWS - 1) / ROWS;
}
template <int TN>
__device__ __forceinline__ int64_t seq_tiles(const Seq& q) {
    return (q.len + TN - 1) / TN;
}

// This CTA's stretch: tiles [begin, end) of row tile rt's line; `begin` lies in
// sequence n, which starts at n_start.
struct Share {
    int64_t begin, end, n_start;
    int rt, n;
    Seq seq;  // of sequence n
};

// Every thread of the CTA takes part (it synchronises the CTA).
template <int ROWS, int TN, int THREADS>
__device__ __forceinline__ Share find_share(const TreeArgs& a) {
    constexpr int W = THREADS / 32;
    __shared__ unsigned long long totals[kMaxRowTiles];
    __shared__ int64_t scan[W], found[2];
    __shared__ Seq found_seq;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = a.p.N, RT = a.row_tiles;
    Share s;
    s.begin = s.end = 0;
    s.rt = RT;
    s.n = N;
    s.n_start = 0;
    auto scan_warp = [&](int64_t x) {  // sum of the warp's values up to this lane's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[warp] = x;
        return x;
    };
    if (RT == 1 && N <= THREADS) {
        // The usual step, a sequence per thread and one line: a single pass. With one
        // sequence of 1021 tokens the way below takes 1.3 us more of the kernel's 7.
        Seq q;
        int64_t own = 0;
        if (tid < N) {
            q = load_seq(a, tid);
            if (q.bad && blockIdx.x == 0) set_status(a.status, kStatusBadSeqlens);
            if (q.nodes > 0) own = a.c.Hk * seq_tiles<TN>(q);
        }
        int64_t start = scan_warp(own) - own;
        __syncthreads();
        int64_t line = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) start += scan[w];
            line += scan[w];
        }
        const int64_t shares = line < (int64_t)gridDim.x ? line : (int64_t)gridDim.x, c = blockIdx.x;
        s.rt = 0;
        if (c < shares) {
            s.begin = quotient(c * line, shares);
            s.end = quotient((c + 1) * line, shares);
            if (start <= s.begin && s.begin < start + own) {
                found[0] = tid;
                found[1] = start;
                found_seq = q;
            }
        }
        __syncthreads();
        if (s.begin == s.end) return s;
        s.n = (int)found[0];
        s.n_start = found[1];
        s.seq = found_seq;
        return s;
    }
    if (tid < RT) totals[tid] = 0;
    if (tid == 0) found[0] = N;
    __syncthreads();
    for (int n = tid; n < N; n += THREADS) {
        const Seq q = load_seq(a, n);
        if (q.bad && blockIdx.x == 0) set_status(a.status, kStatusBadSeqlens);
        const int last = seq_row_tiles<ROWS>(a, q) - 1;
        if (last >= 0) atomicAdd(&totals[last], (unsigned long long)(a.c.Hk * seq_tiles<TN>(q)));
    }
    __syncthreads();
    // line rt holds every sequence with more than rt row tiles
    int64_t all = 0, active = 0, run = 0;
    for (int rt = RT - 1; rt >= 0; --rt) {
        run += (int64_t)totals[rt];
        all += run;
        active += run > 0;
    }
    {
        int64_t line = run;  // line 0
        int cta = 0;
        for (int rt = 0; rt < RT && line > 0; ++rt) {
            const int64_t count = 1 + quotient(((int64_t)gridDim.x - active) * line, all);
            const int64_t shares = line < count ? line : count;
            const int64_t c = (int64_t)blockIdx.x - cta;
            if (c >= 0 && c < shares) {
                s.rt = rt;
                s.begin = quotient(c * line, shares);
                s.end = quotient((c + 1) * line, shares);
            }
            cta += (int)count;
            line -= (int64_t)totals[rt];
        }
    }
    if (s.begin == s.end) return s;
    int64_t before = 0;
    for (int n0 = 0; n0 < N; n0 += THREADS) {
        const int n = n0 + tid;
        int64_t own = 0;
        if (n < N) {
            const Seq q = load_seq(a, n);
            if (seq_row_tiles<ROWS>(a, q) > s.rt) own = a.c.Hk * seq_tiles<TN>(q);
        }
        const int64_t x = scan_warp(own);
        __syncthreads();
        int64_t pre = before;
        for (int w = 0; w < W; ++w) {
            if (w < warp) pre += scan[w];
            before += scan[w];
        }
        const int64_t start = pre + x - own;
        if (start <= s.begin && s.begin < start + own) {
            found[0] = n;
            found[1] = start;
        }
        __syncthreads();
        if (found[0] < N) break;
    }
    s.n = (int)found[0];
    s.n_start = found[1];
    s.seq = load_seq(a, s.n);
    return s;
}

// The part of a CTA's stretch that lies in one unit.
struct Segment {
    Seq seq;
    int n, hk, rt, rows;      // rows: query rows of this row tile
    int tile0, tile1, tiles;  // its token tiles, of the unit's
    int later;                // 0: it starts where the stretch starts
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
    int64_t n_start, end;     // of the sequence and of this segment, on the line
};

template <int ROWS, int TN>
__device__ __forceinline__ void place_segment(const TreeArgs& a, const Share& s, int64_t at, Segment& g) {
    g.tiles = (int)seq_tiles<TN>(g.seq);
    const int64_t unit = quotient(at - g.n_start, g.tiles), unit_start = g.n_start + unit * g.tiles;
    g.hk = (int)unit;
    g.tile0 = (int)(at - unit_start);
    g.tile1 = (int)(s.end - unit_start < g.tiles ? s.end - unit_start : g.tiles);
    g.later = at != s.begin;
    g.rt = s.rt;
    g.rows = min(ROWS, g.seq.nodes * (a.H / a.c.Hk) - s.rt * ROWS);
    g.end = unit_start + g.tile1;
}
template <int ROWS, int TN>
__device__ __forceinline__ bool first_segment(const TreeArgs& a, const Share& s, Segment& g) {
    if (s.begin == s.end) return false;
    g.n = s.n;
    g.n_start = s.n_start;
    g.seq = s.seq;
    place_segment<ROWS, TN>(a, s, s.begin, g);
    return true;
}
template <int ROWS, int TN>
__device__ __forceinline__ bool next_segment(const TreeArgs& a, const Share& s, Segment& g) {
    const int64_t at = g.end;
    if (at >= s.end) return false;
    int64_t len = a.c.Hk * seq_tiles<TN>(g.seq);
    while (at >= g.n_start + len) {  // the next sequence on the line
        g.n_start += len;
        g.seq = load_seq(a, ++g.n);
        len = seq_row_tiles<ROWS>(a, g.seq) > s.rt ? a.c.Hk * seq_tiles<TN>(g.seq) : 0;
    }
    place_segment<ROWS, TN>(a, s, at, g);
    return true;
}

// Tells the joining kernel where a unit's partials are (one thread per segment).
__device__ __forceinline__ void note_parts(const TreeArgs& a, const Segment& g) {
    UnitParts* u = unit_parts(a, g.rt, g.n, g.hk);
    if (g.tile0 == 0) u->first = 2 * (int)blockIdx.x + g.later;
    if (g.tile1 == g.tiles) u->last = (int)blockIdx.x;
}

}  // namespace gdn
