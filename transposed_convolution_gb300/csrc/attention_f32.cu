// attention_f32.cu -- the paged attention's kernels for fp32 caches.
#include "attention_launch.cuh"

namespace ctr {
namespace {

template <int H>
cudaError_t launch32(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    using attn::Heads32;
    using attn::launch;
    switch (p.D) {
    case 64: return launch<Heads32<64, H, 64>>(pl, p, st);
    case 80: return launch<Heads32<96, H, 80>>(pl, p, st);
    case 96: return launch<Heads32<96, H, 96>>(pl, p, st);
    case 128: return launch<Heads32<128, H, 128>>(pl, p, st);
    }
    return p.D < 64    ? launch<Heads32<64, H, 0>>(pl, p, st)
           : p.D < 128 ? launch<Heads32<128, H, 0>>(pl, p, st)
                       : launch<Heads32<256, H, 0>>(pl, p, st);
}

}  // namespace

cudaError_t launch_attention_f32(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    return p.G <= 2 ? launch32<2>(pl, p, st) : launch32<8>(pl, p, st);
}

}  // namespace ctr
