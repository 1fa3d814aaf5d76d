// attention.cu -- the paged attention by type, and the kernel that accumulates its weights.
#include <algorithm>

#include "attention_kernel.cuh"

namespace ctr {
namespace {

// w_out = w_in + the group's probabilities, from the scores and statistics that the attention left: 4 G
// + 8 bytes a slot, of which the scores are mostly still in L2.
__global__ void weights_kernel(AttnParams p, int chunks) {
    const int unit = blockIdx.x / chunks, hk = unit % p.Hkv, b = unit / p.Hkv;
    ptx::griddep_wait();
    const int len = p.cache.lens[b], n = token_count(p.cache, b, p.k_new != nullptr);
    const int lo = attn::first_slot(p, n);
    const int64_t base = ((int64_t)b * p.Hkv + hk) * p.cache.cap, h0 = (int64_t)b * p.Hq + hk * p.G;
    for (int j = blockIdx.x % chunks * blockDim.x + threadIdx.x; j < n; j += chunks * blockDim.x) {
        float w = 0.0f;
        if (j >= lo)
            for (int g = 0; g < p.G; ++g) {
                const float2 st = p.stats[h0 + g];
                if (st.y > 0.0f)
                    w += exp2f(p.scores[(h0 + g) * p.score_pitch + j] - st.x) / st.y;
            }
        p.w_out[base + j] = (p.w_in && j < len ? p.w_in[base + j] : 0.0f) + w;
    }
}

}  // namespace

cudaError_t launch_attention(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    const cudaError_t e = pl->dtype == CTR_F32    ? launch_attention_f32(pl, p, st)
                          : pl->dtype == CTR_BF16 ? launch_attention_bf16(pl, p, st)
                                                  : launch_attention_f16(pl, p, st);
    if (e != cudaSuccess || !p.w_out) return e;
    const int chunks = std::min((p.cache.cap + 1023) / 1024, 64);
    count_launches(1);
    return launch_pdl(weights_kernel, dim3((unsigned)(p.B * p.Hkv) * chunks), dim3(256), 0, st, p, chunks);
}

}  // namespace ctr
