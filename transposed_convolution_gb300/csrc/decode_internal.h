// decode_internal.h -- state and parameter blocks of the decode-step operators (attention over
// a paged cache, eviction, sampling).  Not part of the public ABI.
#pragma once

#include "ctr_internal.h"

struct ctr_attn_s {
    int64_t B, Hq, Hkv, D, page, max_pages;
    int dtype, layout, weights, num_sms;
    int64_t window;
    float scale;
    void *k_pages, *v_pages;
    int64_t num_pages;
    size_t off_parts, off_ml, off_stats, off_scores, ws_needed;
    int64_t score_pitch;
    void *ws;
    size_t ws_bytes;
    int ready;               // ctr_attn_reset ran on the bound workspace
};

namespace ctr {

// Status-word bits of the attention plan (the first word of its workspace).
constexpr uint32_t kStatusBadPage = 1u << 0;
constexpr uint32_t kStatusBadLength = 1u << 1;

// The paged cache as kernels see it: row r of page p of head h is at
// p * page_stride + h * head_stride + r * row_stride elements.
struct CacheView {
    const int32_t *tables;   // [B][table_pitch]
    const int32_t *lens;     // [B]
    int64_t page_stride, head_stride, row_stride;
    int table_pitch, page, num_pages, cap;   // cap: slots of one sequence
    uint32_t *status;
};

struct AttnParams {
    CacheView cache;
    void *k, *v;
    const void *q, *k_new, *v_new;
    int64_t q_stride, kv_stride;
    void *out;
    float *scores;           // [B * Hq][score_pitch] scores in units of log 2, with weights
    float2 *stats;           // [B * Hq] maximum score and sum of the softmax, with weights
    int64_t score_pitch;
    // Parts of units that several chunks of the work share, two to a chunk (its first segment
    // and a later one): [part_rows][D] outputs and [part_rows] (maximum, sum) each.
    float *part_o;
    float2 *part_ml;
    int part_rows;
    int whole_units;         // every chunk is a whole unit: no parts
    int page_shift;          // log2 of the page size, or -1
    const float *w_in;
    float *w_out;
    int B, Hq, Hkv, G, D;
    int64_t window;
    float scale_log2;        // scale * log2(e): scores are kept in units of log 2
};

struct EvictParams {
    CacheView cache;
    void *k, *v;
    const float *w;
    const int32_t *dst_tables;
    int64_t dst_pitch, w_pitch;
    int budget, sinks, recent;
    int32_t *slots, *lens_out;
    float *w_out;
    int B, Hkv, row_bytes, esize, num_sms;
};

// Most blocks an SM that an attention launch has; the workspace holds two parts for each.
constexpr int kMaxPerSm = 4;
// Score rows are padded to whole tiles (64 or 96 slots).
constexpr int kScoreTile = 192;
// Caches of up to this many slots a sequence are cut into whole units.
constexpr int kWholeSlots = 256;

// SMs of the current device (152 without one).
inline int device_sms() {
    const int dev = current_device();
    int n = 0;
    if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    return n > 0 ? n : 152;
}

cudaError_t launch_attention_f32(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention_bf16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention_f16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_evict(const EvictParams &p, cudaStream_t st);

}  // namespace ctr
