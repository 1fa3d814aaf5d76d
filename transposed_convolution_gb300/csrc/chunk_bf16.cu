// chunk_bf16.cu -- the chunk attention of bf16 caches (instantiations of chunk_tc.cuh).
#include "chunk_tc.cuh"

namespace ctr {

cudaError_t launch_chunk_bf16(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    return chunk::launch_16<__nv_bfloat16>(pl, p, st);
}

}  // namespace ctr
