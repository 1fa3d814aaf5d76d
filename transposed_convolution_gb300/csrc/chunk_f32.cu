// chunk_f32.cu -- attention of a chunk of new tokens over a paged fp32 cache.
//
// Two products of 64 rows by 64 slots by D a tile, as fp32 multiply-adds on the CUDA cores, which bound
// it: a thread has 4 x 4 scores and 4 x D / 16 outputs, so that 64 multiply-adds go to eight 16-byte
// loads from shared memory, two an instruction.  6 sequences of 100 to 311 tokens with a window of 750, 16/8
// heads of 80: 164 us (24 TFLOP/s); 512 tokens on 4096, 32/8 heads of 128: 986 us (37).  What keeps it from the
// multiply-adds' rate: one buffer of K and V, so that copies and products take turns; at two blocks an SM
// (128 registers) a few spills (12 to 104 bytes a thread; none where D > 128); and 80 columns are five a thread, an odd
// number, whose second product goes one multiply-add an instruction.  (The tensor pipe's accumulation, even of tf32
// terms that add up to fp32, truncates, which would cost the result digits.)
#include <algorithm>

#include "chunk_device.cuh"
#include "chunk_join.cuh"

namespace ctr {
namespace chunk {

constexpr int kRows = 64, kSlots = 64, kThreads = 256;

// Floats of shared memory: Q and K rows (16-byte reads of eight rows fall into different banks), V rows; P
// takes K's place.
__host__ __device__ constexpr int row_pitch(int D) { return D + 4; }
constexpr int kPPitch = kSlots + 4;
inline size_t smem_bytes(int D, int DP) {
    return sizeof(float) * ((size_t)kRows * row_pitch(D) + std::max(kSlots * row_pitch(D), kRows * kPPitch) +
                            (size_t)kSlots * DP);
}

__device__ __forceinline__ float4 load4(const float *from) { return *reinterpret_cast<const float4 *>(from); }

// NC: columns a thread has, of up to 16 NC.  Thread (ty, tx) has rows 4 ty .. 4 ty + 3, slots tx + 16 j
// and columns tx * 4 + 64 j .. + 3 (tx + 16 c where NC is no multiple of four).
template <int NC> __device__ __forceinline__ int column(int tx, int c) {
    return NC % 4 == 0 ? tx * 4 + c / 4 * 64 + c % 4 : tx + 16 * c;
}

template <int NC> __global__ void __launch_bounds__(kThreads, NC <= 8 ? 2 : 1) chunk_kernel(ChunkParams p) {
    constexpr int DP = 16 * NC;
    extern __shared__ __align__(16) float smem[];
    __shared__ int64_t costs[kMaxB + 1];
    __shared__ Start start;
    __shared__ int visible[kSlots];
    __shared__ int tainted;
    const int D = p.D, pitch = row_pitch(D), t = threadIdx.x, tx = t % 16, ty = t / 16;
    float *const sq = smem, *const sk = sq + kRows * pitch;
    float *const sp = sk, *const sv = sk + max(kSlots * pitch, kRows * kPPitch);
    ptx::griddep_wait();
    sum_costs<kRows, kSlots>(p, costs);
    __syncthreads();
    if (t < 32) {
        const Start s = find_start<kRows, kSlots>(p, costs);
        if (t == 0) start = s;
    }
    __syncthreads();
    Walk<kRows, kSlots> walk;
    walk.start(p, start);
    int4 head = make_int4(0, 0, 0, 0);
    // Columns past D stay zero in V.
    for (int i = t; i < kSlots * (DP - D); i += kThreads) sv[i / (DP - D) * DP + D + i % (DP - D)] = 0.0f;
    while (walk.next(p)) {
        const Unit<kRows, kSlots> &u = walk.u;
        __syncthreads();                 // the segment before is done with Q
        for (int i = t; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float4 x = r < u.rows ? load4((const float *)p.q + query_offset(p, u, r) + d)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(sq + r * pitch + d) = x;
        }
        if (t == 0) tainted = 0;
        int lo[4], hi[4];                // slots that this thread's rows attend to
        float m[4], l[4], o[4][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            hi[i] = r < u.rows ? end_slot(p, u.s, (u.r0 + r) / p.G) : 0;
            lo[i] = first_slot(p, hi[i]);
            m[i] = kNegInf;
            l[i] = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = 0.0f;
        }
        for (int tile = walk.t0; tile < walk.t1; ++tile) {
            const int j0 = (u.first + tile) * kSlots;
            const bool edge = is_edge(u, j0, kSlots);
            __syncthreads();             // the tile before is done with K, V and P
            int hidden = 0;
            {
                // Four threads a slot.
                const int r = t / 4, j = j0 + r;
                const int64_t at = cache_row(p.cache, p.page_shift, u, j);
                hidden = at < 0 && j >= u.lo && j < u.hi;
                if (t % 4 == 0) visible[r] = at >= 0;
                for (int d = t % 4 * 4; d < D; d += 16) {
                    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                    if (at >= 0) {
                        k = load4((const float *)p.k + at + d);
                        v = load4((const float *)p.v + at + d);
                        if (edge && !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) {
                            tainted = 1;
                            v.x = isfinite(v.x) ? v.x : 0.0f;
                            v.y = isfinite(v.y) ? v.y : 0.0f;
                            v.z = isfinite(v.z) ? v.z : 0.0f;
                            v.w = isfinite(v.w) ? v.w : 0.0f;
                        }
                    }
                    *reinterpret_cast<float4 *>(sk + r * pitch + d) = k;
                    *reinterpret_cast<float4 *>(sv + r * DP + d) = v;
                }
            }
            const bool masked = __syncthreads_or(hidden) || edge;
            float s[4][4];
            uint64_t s2[4][4] = {};          // sums over even and over odd columns
            for (int d = 0; d < D; d += 4) {
                ulonglong2 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[i] = *reinterpret_cast<ulonglong2 *>(sq + (ty * 4 + i) * pitch + d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[j] = *reinterpret_cast<ulonglong2 *>(sk + (tx + 16 * j) * pitch + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s2[i][j] = fma2(a[i].x, b[j].x, s2[i][j]);
                        s2[i][j] = fma2(a[i].y, b[j].y, s2[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float even, odd;
                    unpair(s2[i][j], even, odd);
                    s[i][j] = even + odd;
                }
            float shrink[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = kNegInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] *= p.scale_log2;
                    if (masked) {
                        const int at = j0 + tx + 16 * j;
                        if (at < lo[i] || at >= hi[i] || !visible[tx + 16 * j]) s[i][j] = kNegInf;
                    }
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int d = 8; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                top = fmaxf(top, m[i]);
                const float base = top == kNegInf ? 0.0f : top;
                shrink[i] = shrink_of(m[i], base);
                m[i] = top;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = pow2(s[i][j] - base);
                    sum += s[i][j];
                }
                l[i] = l[i] * shrink[i] + sum;
            }
            __syncthreads();             // all have read K
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sp[(ty * 4 + i) * kPPitch + tx + 16 * j] = s[i][j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] *= shrink[i];
            __syncwarp();                // a warp reads the rows that it wrote
            for (int j = 0; j < kSlots; j += 4) {
                float4 a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<float4 *>(sp + (ty * 4 + i) * kPPitch + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float b[NC];
                    if (NC % 4 == 0) {
#pragma unroll
                        for (int c = 0; c < NC / 4; ++c)
                            *reinterpret_cast<float4 *>(b + 4 * c) =
                                *reinterpret_cast<float4 *>(sv + (j + e) * DP + tx * 4 + 64 * c);
                    } else {
#pragma unroll
                        for (int c = 0; c < NC; ++c) b[c] = sv[(j + e) * DP + tx + 16 * c];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
                        if (NC % 2 == 0) {
                            const uint64_t x2 = pair(x, x);
#pragma unroll
                            for (int c = 0; c + 1 < NC; c += 2)
                                unpair(fma2(x2, pair(b[c], b[c + 1]), pair(o[i][c], o[i][c + 1])), o[i][c],
                                       o[i][c + 1]);
                        } else {
#pragma unroll
                            for (int c = 0; c < NC; ++c) o[i][c] = fmaf(x, b[c], o[i][c]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 8; d > 0; d /= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        if (tainted)
            for (int i = 0; i < 4; ++i)
                for (int c = 0; c < NC; ++c)
                    if (column<NC>(tx, c) < D)
                        o[i][c] += taint_of<float, kSlots>(p, u, walk.t0, walk.t1, lo[i], hi[i], column<NC>(tx, c));
        if (walk.part) {
            const int64_t slot = walk.slot();
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (column<NC>(tx, c) < D)
                    *reinterpret_cast<float4 *>(p.part_o + (slot * D + column<NC>(tx, c)) * kRows + ty * 4) =
                        make_float4(o[0][c], o[1][c], o[2][c], o[3][c]);
            if (tx == 0)
                for (int i = 0; i < 4; ++i)
                    p.part_ml[slot * kRows + ty * 4 + i] = make_float2(m[i], l[i]);
            if (walk.begins) head = make_int4(u.b, u.hk, u.m, walk.parts());
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (ty * 4 + i >= u.rows) continue;
                float *to = (float *)p.out + output_offset(p, u, ty * 4 + i);
                // (A row without weight is 0 whatever V holds: 0 times an infinity would be NaN.)
                const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (column<NC>(tx, c) < D) to[column<NC>(tx, c)] = l[i] == 0.0f ? 0.0f : o[i][c] * inv;
            }
        }
    }
    if (t == 0 && !p.whole) p.heads[blockIdx.x] = head;
}

template <int NC> cudaError_t launch(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    static PerDeviceOnce once;
    const auto kernel = chunk_kernel<NC>;
    cudaError_t e = once.run(current_device(), cudaSuccess, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem_bytes(16 * NC, 16 * NC));
    });
    if (e != cudaSuccess) return e;
    const int grid = pl->num_sms * chunk_shape(CTR_F32, pl->D).per_sm;
    count_launches(1);
    e = launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), smem_bytes(p.D, 16 * NC), st, p);
    if (e != cudaSuccess || p.whole) return e;
    return launch_join<float, kRows>(p, grid, st);
}

}  // namespace chunk

cudaError_t launch_chunk_f32(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    using namespace chunk;
    if (p.D <= 64) return launch<4>(pl, p, st);
    if (p.D <= 80) return launch<5>(pl, p, st);
    if (p.D <= 96) return launch<6>(pl, p, st);
    if (p.D <= 128) return launch<8>(pl, p, st);
    return launch<16>(pl, p, st);
}

}  // namespace ctr
