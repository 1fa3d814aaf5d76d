// chunk_device.cuh -- device helpers shared by the chunk attention's kernels.
#pragma once

#include "chunk_schedule.cuh"

namespace ctr {
namespace chunk {

constexpr float kNegInf = -__builtin_inff();

// Two fp32 operations an instruction, which halves what a score costs to issue.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 2^x with a relative error of 2^-22; 0 at -inf.
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a sum whose maximum was m is worth under a larger base: never 0 unless it is empty, so that an infinite
// output stays infinite.
__device__ __forceinline__ float shrink_of(float m, float base) {
    return m == kNegInf ? 0.0f : fmaxf(pow2(m - base), 1.17549435e-38f);
}

// Where row r of a unit is in q and in the output.
template <typename U> __device__ __forceinline__ int64_t query_offset(const ChunkParams &p, const U &u, int r) {
    const int row = u.r0 + r, tok = row / p.G;
    return (u.s.row0 + (int64_t)tok) * p.q_stride + (int64_t)(u.hk * p.G + row - tok * p.G) * p.D;
}
template <typename U> __device__ __forceinline__ int64_t output_offset(const ChunkParams &p, const U &u, int r) {
    const int row = u.r0 + r, tok = row / p.G;
    return ((u.s.row0 + (int64_t)tok) * p.Hq + u.hk * p.G + row - tok * p.G) * p.D;
}

// First element of a unit's slot j, or -1 for slots that no row of it attends to (their pages may
// be gone) and for pages out of range, which are reported.
template <typename U>
__device__ __forceinline__ int64_t cache_row(const CacheView &c, int page_shift, const U &u, int j) {
    if (j < u.lo || j >= u.hi) return -1;
    const int at = page_shift >= 0 ? j >> page_shift : j / c.page;
    const int pg = c.tables[(int64_t)u.b * c.table_pitch + at];
    if ((unsigned)pg >= (unsigned)c.num_pages) {
        atomicOr(c.status, kStatusBadPage);
        return -1;
    }
    return pg * c.page_stride + u.hk * c.head_stride + (int64_t)(j - at * c.page) * c.row_stride;
}

// Whether some row does not attend to all of the slots [j0, j0 + n).
template <typename U> __device__ __forceinline__ bool is_edge(const U &u, int j0, int n) {
    return j0 < u.lo_last || j0 + n > u.hi_first;
}

template <typename T> __device__ __forceinline__ float widen(T v);
template <> __device__ __forceinline__ float widen(float v) { return v; }
template <> __device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float widen(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T round_to(float v);
template <> __device__ __forceinline__ float round_to(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 round_to(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half round_to(float v) { return __float2half_rn(v); }

__device__ __forceinline__ void store8(float *to, const float (&v)[8]) {
    reinterpret_cast<float4 *>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T> __device__ __forceinline__ void store8(T *to, const float (&v)[8]) {
    __align__(16) T x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = round_to<T>(v[i]);
    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<uint4 *>(x);
}

// A tile's products take all its slots for all its rows, and 0 times an infinity or NaN of a slot
// that a row does not attend to would be NaN.  So infinities and NaN are taken out of V in the tiles that
// some row attends to in part, and the unit is marked.  This is what they add to one output: the
// infinities and NaN among the slots [lo, hi) of those tiles of the segment.
// (By value: what has its address taken is in memory from then on.)
struct Edges {
    CacheView cache;
    const void *v;
    int page_shift, b, hk, lo, hi, lo_last, hi_first, first;
};
template <typename T, int NT> __device__ __noinline__ float taint(Edges u, int t0, int t1, int lo, int hi, int d) {
    float sum = 0.0f;
    for (int tile = t0; tile < t1; ++tile) {
        const int j0 = (u.first + tile) * NT;
        if (!is_edge(u, j0, NT)) continue;
        for (int j = max(lo, j0); j < min(hi, j0 + NT); ++j) {
            const int64_t at = cache_row(u.cache, u.page_shift, u, j);
            const float v = at < 0 ? 0.0f : widen(((const T *)u.v)[at + d]);
            if (!isfinite(v)) sum += v;
        }
    }
    return sum;
}
template <typename T, int NT, typename U>
__device__ __forceinline__ float taint_of(const ChunkParams &p, const U &u, int t0, int t1, int lo,
                                          int hi, int d) {
    const Edges e = {p.cache, p.v, p.page_shift, u.b, u.hk, u.lo, u.hi, u.lo_last, u.hi_first, u.first};
    return taint<T, NT>(e, t0, t1, lo, hi, d);
}

}  // namespace chunk
}  // namespace ctr
