// attention_bf16.cu -- the paged attention's kernels for bf16 caches.
#include "attention_launch.cuh"

namespace ctr {

cudaError_t launch_attention_bf16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    return p.G <= 8 ? attn::launch16<__nv_bfloat16, 1>(pl, p, st) : attn::launch16<__nv_bfloat16, 2>(pl, p, st);
}

}  // namespace ctr
