// chunk_f16.cu -- the chunk attention of fp16 caches (instantiations of chunk_tc.cuh).
#include "chunk_tc.cuh"

namespace ctr {

cudaError_t launch_chunk_f16(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    return chunk::launch_16<__half>(pl, p, st);
}

}  // namespace ctr
