// decode_device.cuh -- device helpers shared by the decode-step kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_internal.h"

namespace ctr {

// Tokens of sequence b (slots 0 .. n - 1), with the new one if there is one and room for it.
// Reports a length past the table's capacity, whichever thread asks; every block asks for all sequences,
// so the first one does.
__device__ __forceinline__ int tokens_of(const CacheView &c, int b, bool with_new, int *len) {
    int n = c.lens[b];
    *len = n;
    if (n < 0) return 0;
    if (n > c.cap - (with_new ? 1 : 0)) {
        if (blockIdx.x == 0) atomicOr(c.status, kStatusBadLength);
        *len = min(n, c.cap);
        return *len;
    }
    return n + (with_new ? 1 : 0);
}

// The same count, without the report.
__device__ __forceinline__ int token_count(const CacheView &c, int b, bool with_new) {
    const int n = c.lens[b];
    return n < 0 ? 0 : n > c.cap - (with_new ? 1 : 0) ? min(n, c.cap) : n + (with_new ? 1 : 0);
}

// First element of slot j of sequence b, or -1 when the table names no page of the cache.
__device__ __forceinline__ int64_t slot_offset(const CacheView &c, int b, int h, int j) {
    const int pg = c.tables[(int64_t)b * c.table_pitch + j / c.page];
    if ((unsigned)pg >= (unsigned)c.num_pages) {
        atomicOr(c.status, kStatusBadPage);
        return -1;
    }
    return pg * c.page_stride + h * c.head_stride + (j % c.page) * c.row_stride;
}

}  // namespace ctr
