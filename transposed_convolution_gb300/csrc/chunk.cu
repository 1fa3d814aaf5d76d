// chunk.cu -- the chunk attention by type.
#include "decode_internal.h"

namespace ctr {

// Rows of a tile and blocks an SM, which the workspace has room for (Sizes in chunk_tc.cuh, chunk_f32.cu).
ChunkShape chunk_shape(int dtype, int64_t D) {
    if (dtype == CTR_F32) return {64, D <= 128 ? 2 : 1};
    return {D <= 128 ? 256 : 128, 1};
}

cudaError_t launch_chunk(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    return pl->dtype == CTR_F32    ? launch_chunk_f32(pl, p, st)
           : pl->dtype == CTR_BF16 ? launch_chunk_bf16(pl, p, st)
                                   : launch_chunk_f16(pl, p, st);
}

}  // namespace ctr
