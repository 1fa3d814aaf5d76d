// attention_launch.cuh -- the launch of the paged attention for one arithmetic; each element type is
// instantiated in a translation unit of its own, because the kernels take long to compile.
#pragma once

#include <algorithm>

#include "attention_kernel.cuh"

namespace ctr {
namespace attn {

template <typename C>
cudaError_t launch(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    typedef typename C::Shape Shape;
    static_assert(Shape::kPerSm <= kMaxPerSm && kScoreTile % (16 * Shape::kWarps) == 0, "shape");
    static PerDeviceOnce once;
    const auto kernel = attention_kernel<C>;
    cudaError_t e = once.run(current_device(), cudaSuccess, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem_bytes<C>(C::kMax, 1024));
    });
    if (e != cudaSuccess) return e;
    // Resident blocks: 228 KB an SM, of which a block also takes 1 KB for the system and up to 1 KB
    // of static arrays.  (Large batches' tables of lengths may cost one.)
    const size_t smem = smem_bytes<C>(p.D, p.B);
    const int per_sm = std::max(1, std::min(Shape::kPerSm, (int)(228 * 1024 / (smem + 2048))));
    const int grid = pl->num_sms * per_sm;
    count_launches(1);
    e = launch_pdl(kernel, dim3((unsigned)grid), dim3(32 * Shape::kWarps), smem, st, p);
    if (e != cudaSuccess || p.whole_units) return e;
    // Few heads have many parts each: eight warps join one; else two.
    count_launches(1);
    const int64_t heads = (int64_t)p.B * p.Hq;
    typedef typename C::Element T;
    constexpr int kTile = 16 * Shape::kWarps, kWide = C::kMax > 128 ? 2 : 1;
    if (heads <= 2048)
        return launch_pdl(join_kernel<T, C::kHeads, kTile, kWide, 8>, dim3((unsigned)heads), dim3(256), 0, st,
                          p, grid);
    return launch_pdl(join_kernel<T, C::kHeads, kTile, kWide, 2>, dim3((unsigned)((heads + 3) / 4)), dim3(256),
                      0, st, p, grid);
}

// Common head sizes have kernels of their own, in which every offset is a constant (1.1 to 1.2 times as
// fast); the others share one for each largest size.  (bf16, 16 ragged sequences, 32/8 heads: 27.1 us for 96
// columns, 31.6 for 112, 32.6 for 128; 46.2 for 160 and 48.9 for 192, on the kernel of 256, which takes 53.2.)
template <typename T, int NH>
cudaError_t launch16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    switch (p.D) {
    case 64: return launch<Heads16<T, 64, NH, 64>>(pl, p, st);
    case 80: return launch<Heads16<T, 128, NH, 80>>(pl, p, st);
    case 96: return launch<Heads16<T, 128, NH, 96>>(pl, p, st);
    case 128: return launch<Heads16<T, 128, NH, 128>>(pl, p, st);
    case 256: return launch<Heads16<T, 256, NH, 256>>(pl, p, st);
    }
    return p.D < 64    ? launch<Heads16<T, 64, NH, 0>>(pl, p, st)
           : p.D < 128 ? launch<Heads16<T, 128, NH, 0>>(pl, p, st)
                       : launch<Heads16<T, 256, NH, 0>>(pl, p, st);
}

}  // namespace attn
}  // namespace ctr
