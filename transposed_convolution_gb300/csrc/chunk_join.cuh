// chunk_join.cuh -- joins the parts of units that several blocks of a chunk attention share.
#pragma once

#include "chunk_device.cuh"

namespace ctr {
namespace chunk {

// Joins the parts of the unit that block x of the attention began, thirty-two rows a block: a thread
// has a row and eight columns at a time.  What it reads is mostly in L2.
template <typename T, int MT> __global__ void __launch_bounds__(256) join_kernel(ChunkParams p) {
    ptx::griddep_wait();
    const int4 head = p.heads[blockIdx.x];
    if (head.w == 0) return;
    Unit<MT, 64> u;
    u.b = head.x;
    u.hk = head.y;
    u.m = head.z;
    u.s = sequence_of(p, u.b, false);
    u.tile(p);
    const int r = blockIdx.y * 32 + threadIdx.x % 32;
    if (r >= u.rows) return;
    const int64_t first = 2 * (int64_t)blockIdx.x + 1;
    float M = kNegInf, L = 0.0f;
    for (int i = 0; i < head.w; ++i)
        M = fmaxf(M, p.part_ml[(i == 0 ? first : first - 1 + 2 * i) * MT + r].x);
    const float base = M == kNegInf ? 0.0f : M;
    for (int i = 0; i < head.w; ++i) {
        const float2 ml = p.part_ml[(i == 0 ? first : first - 1 + 2 * i) * MT + r];
        L += ml.y * shrink_of(ml.x, base);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    T *to = (T *)p.out + output_offset(p, u, r);
    for (int d = threadIdx.x / 32 * 8; d < p.D; d += 64) {
        float o[8] = {};
        for (int i = 0; i < head.w; ++i) {
            const int64_t slot = i == 0 ? first : first - 1 + 2 * i;
            const float w = shrink_of(p.part_ml[slot * MT + r].x, base);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += w * p.part_o[(slot * p.D + d + e) * MT + r];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
        store8(to + d, o);
    }
}

template <typename T, int MT> cudaError_t launch_join(const ChunkParams &p, int blocks, cudaStream_t st) {
    count_launches(1);
    return launch_pdl(join_kernel<T, MT>, dim3((unsigned)blocks, MT / 32), dim3(256), 0, st, p);
}

}  // namespace chunk
}  // namespace ctr
