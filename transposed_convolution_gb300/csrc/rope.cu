// rope.cu -- rotary positions (ctr_rope_*), alone or on the way into the cache (ctr_attn_put).
//
// Pair i of a head's first R columns is turned by position * f_i.  Every element is read and written
// once and meets two multiply-adds, so memory bounds it; the sines and cosines, R / 2 a token, are
// computed once a block for the heads it holds, in shared memory.
//
// Angles: a position has up to 31 bits and fp32 only 24, so position * f_i is taken in integers.
// The plan holds f_i / 2 pi, the turns a position makes, as a 64-bit binary fraction; the product with
// the position modulo 2^64 drops whole turns and nothing else, and its upper 32 bits are the
// angle, at most half a turn, in units of 2^-32 turn, of which sincospif() takes the nearest fp32 (within
// 2^-26 turn).  f_i itself is computed in 64 bits, whose 2^-53 a position of 2^22 makes 2^-31 turn.
// A negative position turns backwards, to 2^-32 turn (what is dropped is dropped downwards in either
// direction): with the same magnitude that is the transpose, the gradient's way.
//
// 8192 tokens of 40 heads of 128, bf16: 33 us for 168 MB (5.0 TB/s, 74% of a copy's rate).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

#include "decode_device.cuh"
#include "ptx.cuh"

struct ctr_rope_s {
    int64_t D, R;
    int dtype, layout;
    double base, factor, original, low, high;
    int scaling;
    float magnitude;
    double custom[256];
    int has_custom;
};

namespace ctr {
namespace {

constexpr int kThreads = 256, kMaxPairs = 256;

struct RopeParams {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_stride, kv_stride, qo_stride, ko_stride;
    const int32_t *positions;
    const int64_t *slots;               // with a cache: where K and V go
    CacheView cache;
    void *k_pages, *v_pages;
    int64_t T;
    int Hq, Hk, Hv, D, R, half;         // half: pairs (i, i + R/2), otherwise (2i, 2i + 1)
    int tokens;                         // a block's
    int parts;                          // blocks that share a block's tokens, heads apart
    float magnitude;
    uint64_t turns[kMaxPairs];          // f_i / 2 pi in units of 2^-64
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// N elements that are loaded and stored at once.
template <typename T, int N> struct __align__(sizeof(T) * N) Pack {
    T v[N];
};

// A block has p.tokens tokens and one in p.parts of their heads (of q, then k, then v).  A thread has one
// unit of the heads: N columns and, where pairs are that far apart, their N partners.  N is one
// 16-byte access, or 1 where strides, addresses or R allow no more.  What hides the loads' latency is warps:
// two units at a time took 40 us for the 168 MB below instead of 33, because of their registers.
template <typename T, int N> __global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p) {
    extern __shared__ __align__(16) float2 table[];    // [tokens][R / 2] cosine and sine
    typedef Pack<T, N> P;
    const int pairs = p.R / 2, heads = p.Hq + p.Hk + p.Hv;
    const int64_t t0 = (int64_t)(blockIdx.x / p.parts) * p.tokens;
    const int here = (int)min((int64_t)p.tokens, p.T - t0), part = blockIdx.x % p.parts;
    const int h0 = part * heads / p.parts, own = (part + 1) * heads / p.parts - h0;
    ptx::griddep_wait();
    if (h0 < p.Hq + p.Hk)
        for (int i = threadIdx.x; i < here * pairs; i += kThreads) {
            const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + i / pairs] * p.turns[i % pairs];
            float s, c;
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
            table[i] = make_float2(c * p.magnitude, s * p.magnitude);
        }
    __syncthreads();
    const bool apart = p.half || N == 1;               // partners in a pack of their own
    const int partner = p.half ? pairs : 1, turned = apart ? pairs / N : p.R / N;
    const int units = turned + (p.D - p.R) / N, rows = here * own;
    // A thread keeps its unit and goes through the block's rows (a head of a token each).
    const int span = min(units, kThreads), step = kThreads / span, mine = threadIdx.x / span;
    if (mine >= step) return;
    for (int u = threadIdx.x % span; u < units; u += span) {
        const bool two = apart && u < turned;
        const int col = u >= turned ? p.R + (u - turned) * N : p.half || N > 1 ? u * N : 2 * u;
        int row = 0, at = mine;
        for (int y = mine; y < rows; y += step, at += step) {
            for (; at >= own; at -= own) ++row;
            int h = h0 + at;
            const int64_t t = t0 + row;
            const bool is_v = h >= p.Hq + p.Hk;
            const T *from;
            T *to;
            if (h < p.Hq) {
                from = (const T *)p.q + t * p.q_stride;
                to = (T *)p.q_out + t * p.qo_stride + (int64_t)h * p.D;
            } else {
                h -= is_v ? p.Hq + p.Hk : p.Hq;
                from = is_v ? (const T *)p.v + t * p.kv_stride : (const T *)p.k + t * p.kv_stride;
                if (p.slots) {
                    const int64_t slot = p.slots[t];
                    if (slot < 0) continue;
                    if (slot >= (int64_t)p.cache.num_pages * p.cache.page) {
                        atomicOr(p.cache.status, kStatusBadPage);
                        continue;
                    }
                    // (Most caches have fewer than 2^32 rows, whose division is short.)
                    const int64_t pg = slot >> 32 ? slot / p.cache.page : (uint32_t)slot / (uint32_t)p.cache.page;
                    to = (T *)(is_v ? p.v_pages : p.k_pages) + pg * p.cache.page_stride +
                         h * p.cache.head_stride + (slot - pg * p.cache.page) * p.cache.row_stride;
                } else {
                    to = (T *)p.k_out + t * p.ko_stride + (int64_t)h * p.D;
                }
            }
            from += (int64_t)h * p.D + col;
            to += col;
            P a = *reinterpret_cast<const P *>(from), b = a;
            if (two) b = *reinterpret_cast<const P *>(from + partner);
            if (u < turned && !is_v) {
                const float2 *cs = table + row * pairs + (apart ? u * N : u * N / 2);
                if (apart) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float m = to_f32(a.v[i]), n = to_f32(b.v[i]);
                        a.v[i] = from_f32<T>(m * cs[i].x - n * cs[i].y);
                        b.v[i] = from_f32<T>(m * cs[i].y + n * cs[i].x);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i + 1 < N; i += 2) {
                        const float m = to_f32(a.v[i]), n = to_f32(a.v[i + 1]);
                        a.v[i] = from_f32<T>(m * cs[i / 2].x - n * cs[i / 2].y);
                        a.v[i + 1] = from_f32<T>(m * cs[i / 2].y + n * cs[i / 2].x);
                    }
                }
            }
            *reinterpret_cast<P *>(to) = a;
            if (two) *reinterpret_cast<P *>(to + partner) = b;
        }
    }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The R / 2 frequencies, in radians a position.
void frequencies(const ctr_rope_s *pl, double *f) {
    const double two_pi = 6.283185307179586476925;
    for (int64_t i = 0; i < pl->R / 2; ++i) {
        if (pl->has_custom) {
            f[i] = pl->custom[i];
            continue;
        }
        f[i] = std::pow(pl->base, -2.0 * (double)i / (double)pl->R);
        if (pl->scaling == CTR_ROPE_SCALE_LINEAR) f[i] /= pl->factor;
        if (pl->scaling == CTR_ROPE_SCALE_PARTS) {
            const double turns = pl->original * f[i] / two_pi;
            const double keep = std::min(1.0, std::max(0.0, (turns - pl->low) / (pl->high - pl->low)));
            f[i] = (1.0 - keep) * f[i] / pl->factor + keep * f[i];
        }
    }
}

void set_turns(const ctr_rope_s *pl, RopeParams *p) {
    double f[kMaxPairs];
    frequencies(pl, f);
    for (int64_t i = 0; i < pl->R / 2; ++i) {
        // (The fraction of the absolute value is exact; that of a small negative one, close to 1, would not be.)
        const double x = std::fabs(f[i] / 6.283185307179586476925);
        const double part = x - std::floor(x);             // (NaN where a tiny factor makes f infinite)
        const uint64_t turn = part < 1.0 ? (uint64_t)(part * 18446744073709551616.0) : 0;
        p->turns[i] = f[i] < 0.0 ? 0 - turn : turn;
    }
    p->magnitude = pl->magnitude;
    p->R = (int)pl->R;
    p->half = pl->layout == CTR_ROPE_HALF;
}

template <typename T, int N> cudaError_t launch(RopeParams &p, cudaStream_t st) {
    // Four tokens a block once that fills the SMs twice over; fewer tokens are
    // a block each, and their heads are shared out while SMs are free.
    const int64_t sms = device_sms(), heads = p.Hq + p.Hk + p.Hv;
    p.tokens = p.T >= 8 * sms ? 4 : 1;
    const int64_t groups = (p.T + p.tokens - 1) / p.tokens;
    p.parts = (int)std::max<int64_t>(1, std::min<int64_t>({heads, 2 * sms / groups, 8}));
    count_launches(1);
    return launch_pdl(rope_kernel<T, N>, dim3((unsigned)(groups * p.parts)), dim3(kThreads),
                      (size_t)p.tokens * (p.R / 2) * sizeof(float2), st, p);
}

// One 16-byte access for 4 or 8 elements, if every row and column unit allows it.
template <typename T> cudaError_t launch(RopeParams &p, cudaStream_t st) {
    constexpr int N = 16 / (int)sizeof(T);
    bool wide = p.D % N == 0 && p.R % N == 0 && (!p.half || p.R / 2 % N == 0);
    for (const void *a : {p.q, p.k, p.v, (const void *)p.q_out, (const void *)p.k_out}) wide &= aligned(a, 16);
    for (int64_t s : {p.q_stride, p.kv_stride, p.qo_stride, p.ko_stride}) wide &= s % N == 0;
    return wide ? launch<T, N>(p, st) : launch<T, 1>(p, st);
}

ctr_status launch(int dtype, RopeParams &p, void *stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CTR_F32    ? launch<float>(p, st)
                          : dtype == CTR_BF16 ? launch<__nv_bfloat16>(p, st)
                                              : launch<__half>(p, st);
    return e == cudaSuccess ? CTR_OK : CTR_ERR_CUDA;
}

}  // namespace
}  // namespace ctr

extern "C" {

ctr_status ctr_rope_create(ctr_rope_t *out, int64_t D, int64_t R, int dtype) {
    if (!out) return CTR_ERR_INVALID_ARG;
    *out = nullptr;
    if (dtype != CTR_F32 && dtype != CTR_BF16 && dtype != CTR_F16) return CTR_ERR_INVALID_ARG;
    if (D < 2 || R < 2 || R > D || R % 2) return CTR_ERR_INVALID_ARG;
    if (D > 2 * ctr::kMaxPairs) return CTR_ERR_UNSUPPORTED;
    ctr_rope_s *pl = new (std::nothrow) ctr_rope_s();
    if (!pl) return CTR_ERR_INVALID_ARG;
    pl->D = D;
    pl->R = R;
    pl->dtype = dtype;
    pl->layout = CTR_ROPE_HALF;
    pl->base = 10000.0;
    pl->magnitude = 1.0f;
    *out = pl;
    return CTR_OK;
}

ctr_status ctr_rope_set_layout(ctr_rope_t pl, int layout) {
    if (!pl || (layout != CTR_ROPE_HALF && layout != CTR_ROPE_INTERLEAVED)) return CTR_ERR_INVALID_ARG;
    pl->layout = layout;
    return CTR_OK;
}

ctr_status ctr_rope_set_base(ctr_rope_t pl, double base) {
    if (!pl || !std::isfinite(base) || base < 1.0) return CTR_ERR_INVALID_ARG;
    pl->base = base;
    pl->has_custom = 0;
    return CTR_OK;
}

ctr_status ctr_rope_set_scaling(ctr_rope_t pl, int scaling, double factor, double original, double low,
                                double high) {
    if (!pl || scaling < CTR_ROPE_SCALE_NONE || scaling > CTR_ROPE_SCALE_PARTS) return CTR_ERR_INVALID_ARG;
    if (scaling != CTR_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor <= 0.0)) return CTR_ERR_INVALID_ARG;
    if (scaling == CTR_ROPE_SCALE_PARTS &&
        (!std::isfinite(original) || original <= 0.0 || !std::isfinite(low) || !std::isfinite(high) ||
         low < 0.0 || high <= low))
        return CTR_ERR_INVALID_ARG;
    pl->scaling = scaling;
    pl->factor = factor;
    pl->original = original;
    pl->low = low;
    pl->high = high;
    pl->has_custom = 0;
    return CTR_OK;
}

ctr_status ctr_rope_set_magnitude(ctr_rope_t pl, float magnitude) {
    if (!pl || !std::isfinite(magnitude)) return CTR_ERR_INVALID_ARG;
    pl->magnitude = magnitude;
    return CTR_OK;
}

ctr_status ctr_rope_set_frequencies(ctr_rope_t pl, const double *f, int64_t n) {
    if (!pl || !f || n != pl->R / 2) return CTR_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i)
        if (!std::isfinite(f[i])) return CTR_ERR_INVALID_ARG;
    std::copy(f, f + n, pl->custom);
    pl->has_custom = 1;
    return CTR_OK;
}

ctr_status ctr_rope_frequencies(ctr_rope_t pl, double *f, int64_t n) {
    if (!pl || !f || n != pl->R / 2) return CTR_ERR_INVALID_ARG;
    ctr::frequencies(pl, f);
    return CTR_OK;
}

ctr_status ctr_rope_forward(ctr_rope_t pl, const void *q, int64_t q_stride, int64_t H_q, const void *k,
                            int64_t k_stride, int64_t H_k, const int32_t *positions, int64_t T, void *q_out,
                            int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
    if (!pl || T < 0 || H_q < 0 || H_k < 0) return CTR_ERR_INVALID_ARG;
    if (T > ((int64_t)1 << 24) || H_q > ((int64_t)1 << 14) || H_k > ((int64_t)1 << 14))
        return CTR_ERR_UNSUPPORTED;
    if (T == 0 || H_q + H_k == 0) return CTR_OK;
    if (!positions || (H_q && (!q || !q_out || q_stride < H_q * pl->D || q_out_stride < H_q * pl->D)) ||
        (H_k && (!k || !k_out || k_stride < H_k * pl->D || k_out_stride < H_k * pl->D)))
        return CTR_ERR_INVALID_ARG;
    const uintptr_t size = pl->dtype == CTR_F32 ? 4 : 2;
    if (!ctr::aligned(positions, 4) || (H_q && (!ctr::aligned(q, size) || !ctr::aligned(q_out, size))) ||
        (H_k && (!ctr::aligned(k, size) || !ctr::aligned(k_out, size))))
        return CTR_ERR_MISALIGNED;
    ctr::RopeParams p = {};
    ctr::set_turns(pl, &p);
    if (H_q) {
        p.q = q;
        p.q_out = q_out;
        p.q_stride = q_stride;
        p.qo_stride = q_out_stride;
        p.Hq = (int)H_q;
    }
    if (H_k) {
        p.k = k;
        p.k_out = k_out;
        p.kv_stride = k_stride;
        p.ko_stride = k_out_stride;
        p.Hk = (int)H_k;
    }
    p.D = (int)pl->D;
    p.positions = positions;
    p.T = T;
    return ctr::launch(pl->dtype, p, stream);
}

ctr_status ctr_attn_put(ctr_attn_t pl, ctr_rope_t rope, const void *q, int64_t q_stride, const void *k,
                        const void *v, int64_t kv_stride, const int32_t *positions, const int64_t *slots,
                        int64_t T, void *q_out, int64_t q_out_stride, void *stream) {
    if (!pl || T < 0 || !q != !q_out || (q && !rope) || (rope && (rope->D != pl->D || rope->dtype != pl->dtype)))
        return CTR_ERR_INVALID_ARG;
    if (T > ((int64_t)1 << 24)) return CTR_ERR_UNSUPPORTED;
    if (T > 0 && (!k || !v || !slots || kv_stride < pl->Hkv * pl->D || (rope && !positions) ||
                  (q && (q_stride < pl->Hq * pl->D || q_out_stride < pl->Hq * pl->D))))
        return CTR_ERR_INVALID_ARG;
    const int64_t size = pl->dtype == CTR_F32 ? 4 : 2;
    for (const void *a : {q, k, v, (const void *)q_out})
        if (!ctr::aligned(a, 16)) return CTR_ERR_MISALIGNED;
    if (!ctr::aligned(positions, 4) || !ctr::aligned(slots, 8) || kv_stride * size % 16 ||
        (q && (q_stride * size % 16 || q_out_stride * size % 16)))
        return CTR_ERR_MISALIGNED;
    if (!pl->k_pages) return CTR_ERR_NOT_PREPARED;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    if (!pl->ready) return CTR_ERR_NOT_PREPARED;
    if (T == 0) return CTR_OK;
    ctr::RopeParams p = {};
    if (rope) ctr::set_turns(rope, &p);
    if (q) {
        p.q = q;
        p.q_out = q_out;
        p.q_stride = q_stride;
        p.qo_stride = q_out_stride;
        p.Hq = (int)pl->Hq;
    }
    p.k = k;
    p.v = v;
    p.kv_stride = kv_stride;
    p.Hk = p.Hv = (int)pl->Hkv;
    p.D = (int)pl->D;
    p.positions = positions;
    p.slots = slots;
    p.cache = ctr::cache_view(pl, nullptr, nullptr);
    p.k_pages = pl->k_pages;
    p.v_pages = pl->v_pages;
    p.T = T;
    return ctr::launch(pl->dtype, p, stream);
}

ctr_status ctr_rope_describe(ctr_rope_t pl, char *buf, size_t len) {
    if (!pl || !buf || len == 0) return CTR_ERR_INVALID_ARG;
    static const char *names[] = {"f32", "bf16", "f16"}, *scalings[] = {"none", "linear", "parts"};
    if (pl->has_custom)
        snprintf(buf, len, "rope %s D=%lld R=%lld %s own frequencies magnitude=%g", names[pl->dtype],
                 (long long)pl->D, (long long)pl->R, pl->layout == CTR_ROPE_HALF ? "half" : "interleaved",
                 pl->magnitude);
    else
        snprintf(buf, len, "rope %s D=%lld R=%lld %s base=%g scaling=%s magnitude=%g", names[pl->dtype],
                 (long long)pl->D, (long long)pl->R, pl->layout == CTR_ROPE_HALF ? "half" : "interleaved",
                 pl->base, scalings[pl->scaling], pl->magnitude);
    return CTR_OK;
}

void ctr_rope_destroy(ctr_rope_t pl) { delete pl; }

}  // extern "C"
