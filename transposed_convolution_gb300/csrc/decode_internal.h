// decode_internal.h -- state and parameter blocks of the decode-step operators (attention over
// a paged cache, eviction, sampling).  Not part of the public ABI.
#pragma once

#include "ctr_internal.h"

struct ctr_attn_s {
    int64_t B, Hq, Hkv, D, page, max_pages;
    int dtype, layout, weights, chunks, num_sms;
    int64_t window;
    float scale;
    void *k_pages, *v_pages;
    int64_t num_pages;
    size_t off_parts, off_ml, off_stats, off_scores, ws_needed;
    size_t off_chunk_o, off_chunk_ml, off_chunk_heads;
    int64_t score_pitch;
    void *ws;
    size_t ws_bytes;
    int ready;               // ctr_attn_reset ran on the bound workspace
    uint64_t wait_limit_ns;
};

namespace ctr {

// Status-word bits of the attention and page plans (the first word of their workspaces).
constexpr uint32_t kStatusBadPage = 1u << 0;
constexpr uint32_t kStatusBadLength = 1u << 1;
constexpr uint32_t kStatusTimeout = 1u << 2;

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

struct ChunkParams {
    CacheView cache;
    const void *k, *v, *q;
    int64_t q_stride, T;
    const int32_t *starts;   // [B + 1]
    void *out;
    // Parts of units that several blocks share, two to a block: [D][rows of a tile] outputs and [rows of
    // a tile] (base, sum), and of each block the unit whose first part it has (sequence, head, tile of
    // rows, parts; none: 0 parts).
    float *part_o;
    float2 *part_ml;
    int4 *heads;
    int B, Hq, Hkv, G, D;
    int64_t window;
    float scale_log2;
    int page_shift;          // log2 of the page size, or -1
    int whole;               // units are not cut
    uint64_t wait_limit_ns;  // of a role's wait for another
};

// A chunk attention's launch: rows of a tile, and blocks an SM.
struct ChunkShape {
    int rows, per_sm;
};
ChunkShape chunk_shape(int dtype, int64_t D);

// Default limit of a role's wait for another in the chunk attention: a unit of 2^28 slots takes 6 s.
constexpr uint64_t kChunkWaitLimitNs = 10000000000;

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

// log2 of a page size, or -1.
inline int page_shift(int64_t page) {
    for (int s = 0; s < 29; ++s)
        if (page == (int64_t)1 << s) return s;
    return -1;
}

// The cache that a plan is bound to, as kernels see it.
inline CacheView cache_view(const ctr_attn_s *pl, const int32_t *tables, const int32_t *lens) {
    CacheView c = {};
    c.tables = tables;
    c.lens = lens;
    c.page_stride = pl->Hkv * pl->page * pl->D;
    c.head_stride = pl->layout == CTR_CACHE_HEAD_MAJOR ? pl->page * pl->D : pl->D;
    c.row_stride = pl->layout == CTR_CACHE_HEAD_MAJOR ? pl->D : pl->Hkv * pl->D;
    c.table_pitch = (int)pl->max_pages;
    c.page = (int)pl->page;
    c.num_pages = (int)pl->num_pages;
    c.cap = (int)(pl->max_pages * pl->page);
    c.status = static_cast<uint32_t *>(pl->ws);
    return c;
}

// Waits for the stream, then reads and clears a plan's status word.
inline ctr_status check_status(void *word, cudaStream_t st) {
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, word, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return CTR_ERR_CUDA;
    if (!v) return CTR_OK;
    if (cudaMemsetAsync(word, 0, sizeof v, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return CTR_ERR_CUDA;
    return v & kStatusTimeout ? CTR_ERR_DEVICE_TIMEOUT : CTR_ERR_INVALID_ARG;
}

cudaError_t launch_attention_f32(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention_bf16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention_f16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_attention(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st);
cudaError_t launch_chunk_f32(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk_bf16(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk_f16(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_chunk(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st);
cudaError_t launch_evict(const EvictParams &p, cudaStream_t st);

}  // namespace ctr
