// attention_f16.cu -- the paged attention's kernels for fp16 caches.
#include "attention_launch.cuh"

namespace ctr {

cudaError_t launch_attention_f16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    return p.G <= 8 ? attn::launch16<__half, 1>(pl, p, st) : attn::launch16<__half, 2>(pl, p, st);
}

}  // namespace ctr
