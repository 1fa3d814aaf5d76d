// chunk_join.cuh -- joins the parts of units that several blocks of a chunk attention share.
#pragma once

#include "chunk_device.cuh"

namespace ctr {
namespace chunk {

// Joins the parts of the unit that block x of the attention began: a warp has thirty-two rows and eight
// columns, and takes the parts four at a time, so that it has 32 loads in flight.  What it reads is in L2.
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
    const int r = blockIdx.y * 32 + threadIdx.x % 32, d = blockIdx.z * 64 + threadIdx.x / 32 * 8;
    if (r >= u.rows || d >= p.D) return;
    // The first part is its block's second, the others are their blocks' first.
    const int64_t first = 2 * (int64_t)blockIdx.x;
    float base = kNegInf, l = 0.0f, o[8] = {};
    for (int i0 = 0; i0 < head.w; i0 += 4) {
        float2 ml[4];
        float v[4][8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = min(i0 + e, head.w - 1);
            const int64_t slot = first + (i == 0 ? 1 : 2 * i);
            ml[e] = p.part_ml[slot * MT + r];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[e][c] = p.part_o[(slot * p.D + d + c) * MT + r];
        }
        float top = base;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i0 + e < head.w) top = fmaxf(top, ml[e].x);
        // (Parts of nothing weigh 0, which keeps a sum that is NaN.)
        const float old = shrink_of(base, top), at = top == kNegInf ? 0.0f : top;
        base = top;
        l *= old;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] *= old;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i0 + e >= head.w) break;
            const float w = shrink_of(ml[e].x, at);
            l += w * ml[e].y;
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] += w * v[e][c];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = l == 0.0f ? 0.0f : o[c] * inv;
    store8((T *)p.out + output_offset(p, u, r) + d, o);
}

template <typename T, int MT> cudaError_t launch_join(const ChunkParams &p, int blocks, cudaStream_t st) {
    count_launches(1);
    return launch_pdl(join_kernel<T, MT>, dim3((unsigned)blocks, MT / 32, (p.D + 63) / 64), dim3(256), 0, st, p);
}

}  // namespace chunk
}  // namespace ctr
