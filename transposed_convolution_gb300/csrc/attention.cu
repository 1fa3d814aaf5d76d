// attention.cu -- the paged attention by type, and the kernel that accumulates its weights.
#include <algorithm>

#include "attention_kernel.cuh"

namespace ctr {
namespace {

// w_out = w_in + the group's probabilities, from the scores and statistics that the attention left: 4 G
// + 8 bytes a slot, of which the scores are mostly still in L2.  A thread takes four slots, a block
// four times its threads of one (sequence, KV head).
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(AttnParams p, int blocks_a_unit) {
    __shared__ float2 stats[128];            // maximum and 1 / sum of each of the group's heads
    const int unit = blockIdx.x / blocks_a_unit, hk = unit % p.Hkv, b = unit / p.Hkv, t = threadIdx.x;
    const int j0 = (blockIdx.x % blocks_a_unit * kWeightThreads + t) * 4;
    ptx::griddep_wait();
    const int len = p.cache.lens[b], n = token_count(p.cache, b, p.k_new != nullptr);
    if (blockIdx.x % blocks_a_unit * kWeightThreads * 4 >= n) return;
    const int lo = attn::first_slot(p, n);
    const int64_t base = ((int64_t)b * p.Hkv + hk) * p.cache.cap + j0, h0 = (int64_t)b * p.Hq + hk * p.G;
    for (int g = t; g < p.G; g += kWeightThreads) {
        const float2 s = p.stats[h0 + g];
        // A head that attends to nothing has no probabilities: 2^(x - inf) = 0.  One whose sum is NaN has
        // nothing but NaN.
        stats[g] = s.y == 0.0f ? make_float2(__builtin_inff(), 0.0f) : make_float2(s.x, 1.0f / s.y);
    }
    // Slots before the window hold no scores of this call; those past the end stay as they are.
    float old[4], w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) old[e] = p.w_in && j0 + e < min(len, n) ? p.w_in[base + e] : 0.0f;
    __syncthreads();
    if (j0 >= n) return;
    if (j0 + 3 >= lo) {
        const float *s = p.scores + h0 * p.score_pitch + j0;
#pragma unroll 4
        for (int g = 0; g < p.G; ++g) {
            const float4 x = *reinterpret_cast<const float4 *>(s + g * p.score_pitch);
            const float2 st = stats[g];
            w[0] += exp2f(x.x - st.x) * st.y;
            w[1] += exp2f(x.y - st.x) * st.y;
            w[2] += exp2f(x.z - st.x) * st.y;
            w[3] += exp2f(x.w - st.x) * st.y;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j0 + e < n) p.w_out[base + e] = old[e] + (j0 + e >= lo ? w[e] : 0.0f);
}

}  // namespace

cudaError_t launch_attention(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    const cudaError_t e = pl->dtype == CTR_F32    ? launch_attention_f32(pl, p, st)
                          : pl->dtype == CTR_BF16 ? launch_attention_bf16(pl, p, st)
                                                  : launch_attention_f16(pl, p, st);
    if (e != cudaSuccess || !p.w_out) return e;
    const int blocks = (p.cache.cap + 4 * kWeightThreads - 1) / (4 * kWeightThreads);
    count_launches(1);
    return launch_pdl(weights_kernel, dim3((unsigned)(p.B * p.Hkv) * blocks), dim3(kWeightThreads), 0, st, p,
                      blocks);
}

}  // namespace ctr
