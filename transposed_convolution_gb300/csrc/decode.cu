// decode.cu -- C ABI of the attention plan: validation, workspace layout and the launches of
// ctr_attn_forward and ctr_attn_evict (kernels in attention.cu and evict.cu).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

#include "decode_internal.h"

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int esize_of(const ctr_attn_s *pl) { return pl->dtype == CTR_F32 ? 4 : 2; }

int part_rows(const ctr_attn_s *pl) { return (int)std::min<int64_t>(16, pl->Hq / pl->Hkv); }

// The status word (cleared by ctr_attn_reset), the parts of shared units, and with
// weights the softmax statistics and scores.
void layout_workspace(ctr_attn_s *pl) {
    const int64_t parts = 2 * ctr::kMaxPerSm * (int64_t)pl->num_sms;
    pl->score_pitch = (pl->max_pages * pl->page + ctr::kScoreTile - 1) / ctr::kScoreTile * ctr::kScoreTile;
    pl->off_parts = 256;
    pl->off_ml = pl->off_parts + align256((size_t)(parts * part_rows(pl) * pl->D) * sizeof(float));
    pl->off_stats = pl->off_ml + align256((size_t)(parts * part_rows(pl)) * sizeof(float2));
    pl->ws_needed = pl->off_stats;
    pl->off_scores = pl->off_stats;
    if (pl->weights) {
        pl->off_scores += align256((size_t)(pl->B * pl->Hq) * sizeof(float2));
        pl->ws_needed = pl->off_scores +
                        (size_t)(pl->B * pl->Hq) * (size_t)pl->score_pitch * sizeof(float);
    }
    pl->ws = nullptr;
    pl->ws_bytes = 0;
    pl->ready = 0;
}

ctr::CacheView cache_view(const ctr_attn_s *pl, const int32_t *tables, const int32_t *lens) {
    ctr::CacheView c = {};
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

}  // namespace

extern "C" {

ctr_status ctr_attn_create(ctr_attn_t *out, int64_t B, int64_t H_q, int64_t H_kv, int64_t D,
                           int64_t page_size, int64_t max_pages, int dtype) {
    if (!out) return CTR_ERR_INVALID_ARG;
    *out = nullptr;
    if (dtype != CTR_F32 && dtype != CTR_BF16 && dtype != CTR_F16) return CTR_ERR_INVALID_ARG;
    if (B < 1 || H_q < 1 || H_kv < 1 || D < 1 || page_size < 1 || max_pages < 1 || H_q % H_kv)
        return CTR_ERR_INVALID_ARG;
    const int64_t cap = (int64_t)1 << 28;
    if (B > 1024 || H_kv > ((int64_t)1 << 20) / B || H_q / H_kv > 128 || D > 256 || D % 16 ||
        page_size > cap || max_pages > cap / page_size ||
        B * H_kv * ((H_q / H_kv + 7) / 8) > ((int64_t)1 << 36) / (page_size * max_pages))
        return CTR_ERR_UNSUPPORTED;
    ctr_attn_s *pl = new (std::nothrow) ctr_attn_s();
    if (!pl) return CTR_ERR_INVALID_ARG;
    pl->B = B;
    pl->Hq = H_q;
    pl->Hkv = H_kv;
    pl->D = D;
    pl->page = page_size;
    pl->max_pages = max_pages;
    pl->dtype = dtype;
    pl->layout = CTR_CACHE_HEAD_MAJOR;
    pl->scale = (float)(1.0 / std::sqrt((double)D));
    pl->num_sms = ctr::device_sms();
    layout_workspace(pl);
    *out = pl;
    return CTR_OK;
}

ctr_status ctr_attn_set_layout(ctr_attn_t pl, int layout) {
    if (!pl || (layout != CTR_CACHE_HEAD_MAJOR && layout != CTR_CACHE_TOKEN_MAJOR))
        return CTR_ERR_INVALID_ARG;
    pl->layout = layout;
    return CTR_OK;
}

ctr_status ctr_attn_set_scale(ctr_attn_t pl, float scale) {
    if (!pl || !std::isfinite(scale)) return CTR_ERR_INVALID_ARG;
    pl->scale = scale;
    return CTR_OK;
}

ctr_status ctr_attn_set_window(ctr_attn_t pl, int64_t window) {
    if (!pl || window < 0) return CTR_ERR_INVALID_ARG;
    pl->window = window;
    return CTR_OK;
}

ctr_status ctr_attn_set_weights(ctr_attn_t pl, int enable) {
    if (!pl || (enable != 0 && enable != 1)) return CTR_ERR_INVALID_ARG;
    pl->weights = enable;
    layout_workspace(pl);
    return CTR_OK;
}

size_t ctr_attn_workspace_bytes(ctr_attn_t pl) { return pl ? pl->ws_needed : 0; }

ctr_status ctr_attn_bind_workspace(ctr_attn_t pl, void *ws, size_t bytes) {
    if (!pl || !ws) return CTR_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return CTR_ERR_MISALIGNED;
    if (bytes < pl->ws_needed) return CTR_ERR_NO_WORKSPACE;
    pl->ws = ws;
    pl->ws_bytes = bytes;
    pl->ready = 0;
    return CTR_OK;
}

ctr_status ctr_attn_reset(ctr_attn_t pl, void *stream) {
    if (!pl) return CTR_ERR_INVALID_ARG;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    if (cudaMemsetAsync(pl->ws, 0, pl->off_parts, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return CTR_ERR_CUDA;
    pl->ready = 1;
    return CTR_OK;
}

ctr_status ctr_attn_bind_cache(ctr_attn_t pl, void *k_pages, void *v_pages, int64_t num_pages) {
    if (!pl || !k_pages || !v_pages || num_pages < 1) return CTR_ERR_INVALID_ARG;
    // Kernels hold row offsets in sixteens of elements in 32 bits (2^37 bytes of 16-bit pages).
    if (num_pages > 0x7fffffff || num_pages > (((int64_t)1 << 32) - 1) / (pl->Hkv * pl->page * (pl->D / 16)))
        return CTR_ERR_UNSUPPORTED;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16)) return CTR_ERR_MISALIGNED;
    pl->k_pages = k_pages;
    pl->v_pages = v_pages;
    pl->num_pages = num_pages;
    return CTR_OK;
}

ctr_status ctr_attn_forward(ctr_attn_t pl, const void *q, int64_t q_stride, const void *k_new,
                            const void *v_new, int64_t kv_stride, const int32_t *tables,
                            const int32_t *lens, const float *weights_in, float *weights_out,
                            void *out, void *stream) {
    if (!pl || !q || !tables || !lens || !out || !k_new != !v_new) return CTR_ERR_INVALID_ARG;
    if (q_stride < pl->Hq * pl->D || (k_new && kv_stride < pl->Hkv * pl->D))
        return CTR_ERR_INVALID_ARG;
    if (pl->weights ? !weights_out : (weights_in || weights_out)) return CTR_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(out, 16) ||
        !aligned(tables, 4) || !aligned(lens, 4) || !aligned(weights_in, 4) ||
        !aligned(weights_out, 4) || q_stride * esize_of(pl) % 16 ||
        (k_new && kv_stride * esize_of(pl) % 16))
        return CTR_ERR_MISALIGNED;
    if (!pl->k_pages) return CTR_ERR_NOT_PREPARED;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    if (!pl->ready) return CTR_ERR_NOT_PREPARED;
    ctr::AttnParams p = {};
    p.cache = cache_view(pl, tables, lens);
    p.k = pl->k_pages;
    p.v = pl->v_pages;
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_stride = q_stride;
    p.kv_stride = kv_stride;
    p.out = out;
    char *ws = static_cast<char *>(pl->ws);
    p.part_o = reinterpret_cast<float *>(ws + pl->off_parts);
    p.part_ml = reinterpret_cast<float2 *>(ws + pl->off_ml);
    p.part_rows = part_rows(pl);
    if (pl->weights) {
        p.stats = reinterpret_cast<float2 *>(ws + pl->off_stats);
        p.scores = reinterpret_cast<float *>(ws + pl->off_scores);
    }
    p.whole_units = pl->max_pages * pl->page <= ctr::kWholeSlots;
    p.score_pitch = pl->score_pitch;
    p.page_shift = -1;
    for (int s = 0; s < 29; ++s)
        if (pl->page == (int64_t)1 << s) p.page_shift = s;
    p.w_in = weights_in;
    p.w_out = weights_out;
    p.B = (int)pl->B;
    p.Hq = (int)pl->Hq;
    p.Hkv = (int)pl->Hkv;
    p.G = (int)(pl->Hq / pl->Hkv);
    p.D = (int)pl->D;
    p.window = pl->window;
    p.scale_log2 = (float)((double)pl->scale * 1.4426950408889634);
    return ctr::launch_attention(pl, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? CTR_OK : CTR_ERR_CUDA;
}

ctr_status ctr_attn_evict(ctr_attn_t pl, const int32_t *tables, const int32_t *lens,
                          const float *weights, const int32_t *dst_tables, int64_t dst_pitch,
                          int64_t budget, int64_t sinks, int64_t recent, int32_t *slots,
                          int32_t *lens_out, float *weights_out, int64_t weights_pitch,
                          void *stream) {
    if (!pl || !tables || !lens || !weights || !dst_tables || !slots || !lens_out ||
        lens_out == lens || weights_out == weights)
        return CTR_ERR_INVALID_ARG;
    if (budget < 1 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return CTR_ERR_INVALID_ARG;
    if (budget > ((int64_t)1 << 28)) return CTR_ERR_UNSUPPORTED;
    if (dst_pitch < (budget + pl->page - 1) / pl->page || (weights_out && weights_pitch < budget))
        return CTR_ERR_INVALID_ARG;
    if (!aligned(tables, 4) || !aligned(lens, 4) || !aligned(weights, 4) || !aligned(dst_tables, 4) ||
        !aligned(slots, 4) || !aligned(lens_out, 4) || !aligned(weights_out, 4))
        return CTR_ERR_MISALIGNED;
    if (!pl->k_pages) return CTR_ERR_NOT_PREPARED;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    if (!pl->ready) return CTR_ERR_NOT_PREPARED;
    ctr::EvictParams p = {};
    p.cache = cache_view(pl, tables, lens);
    p.k = pl->k_pages;
    p.v = pl->v_pages;
    p.w = weights;
    p.dst_tables = dst_tables;
    p.dst_pitch = dst_pitch;
    p.w_pitch = weights_pitch;
    p.budget = (int)budget;
    p.sinks = (int)sinks;
    p.recent = (int)recent;
    p.slots = slots;
    p.lens_out = lens_out;
    p.w_out = weights_out;
    p.B = (int)pl->B;
    p.Hkv = (int)pl->Hkv;
    p.esize = esize_of(pl);
    p.num_sms = pl->num_sms;
    p.row_bytes = (int)pl->D * p.esize;
    return ctr::launch_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CTR_OK
                                                                                 : CTR_ERR_CUDA;
}

ctr_status ctr_attn_check(ctr_attn_t pl, void *stream) {
    if (!pl) return CTR_ERR_INVALID_ARG;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    if (!pl->ready) return CTR_ERR_NOT_PREPARED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, pl->ws, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return CTR_ERR_CUDA;
    if (!v) return CTR_OK;
    if (cudaMemsetAsync(pl->ws, 0, sizeof v, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return CTR_ERR_CUDA;
    return CTR_ERR_INVALID_ARG;
}

ctr_status ctr_attn_describe(ctr_attn_t pl, char *buf, size_t len) {
    if (!pl || !buf || len == 0) return CTR_ERR_INVALID_ARG;
    static const char *names[] = {"f32", "bf16", "f16"};
    snprintf(buf, len, "attention %s B=%lld Hq=%lld Hkv=%lld D=%lld page=%lld max_pages=%lld %s "
             "window=%lld weights=%d ws=%zu", names[pl->dtype], (long long)pl->B, (long long)pl->Hq,
             (long long)pl->Hkv, (long long)pl->D, (long long)pl->page, (long long)pl->max_pages,
             pl->layout == CTR_CACHE_HEAD_MAJOR ? "head-major" : "token-major",
             (long long)pl->window, pl->weights, pl->ws_needed);
    return CTR_OK;
}

void ctr_attn_destroy(ctr_attn_t pl) { delete pl; }

}  // extern "C"
