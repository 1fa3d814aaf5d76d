// sampler.cu -- sampling with temperature, top-k, top-p and min-p from given random numbers.
#include <cstdio>
#include <new>

#include "decode_device.cuh"

struct ctr_sampler_s {
    int64_t rows, vocab;
    int dtype;
};

namespace ctr {
namespace {

constexpr int kThreads = 512;

struct SampleParams {
    const void *logits;
    const float *noise;
    int64_t logits_stride, noise_stride;
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *tokens;
    int vocab;
};

// Order-preserving key of a logit (NaN as -inf, -0 as +0) and back.
__device__ __forceinline__ uint32_t logit_key(float l) {
    if (l != l) l = -__builtin_inff();
    const uint32_t u = __float_as_uint(l + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// w_i = exp((l - m) / T), 1 at the maximum (also when it is infinite).
__device__ __forceinline__ float weight_of(float l, float m, float T) {
    return l == m ? 1.0f : expf((l - m) / T);
}
// Masses are sums of weights (at most 1, up to 2^20 of them) in units of 2^-40.
__device__ __forceinline__ unsigned long long fixed_of(float w) {
    return __float2ull_rn(w * 1099511627776.0f);
}

template <typename V, typename F>
__device__ V block_reduce(V v, V *red, F f) {
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i) v = f(v, red[i]);
    return v;
}

// One block a row.  Every filter keeps a prefix of the order (logit descending, index
// ascending), so the kept set is: keys above `cut`, and the first `ties` tokens with key `cut`.
template <typename T>
__global__ void sample_kernel(SampleParams p) {
    typedef unsigned long long u64;
    __shared__ u64 red[kThreads / 32];
    const int row = blockIdx.x, t = threadIdx.x, V = p.vocab;
    const T *logits = static_cast<const T *>(p.logits) + row * p.logits_stride;
    const float *noise = p.noise + row * p.noise_stride;
    auto key = [&](int i) { return logit_key(to_f(logits[i])); };
    auto sum = [](u64 a, u64 b) { return a + b; };
    auto most = [](u64 a, u64 b) { return a > b ? a : b; };

    u64 top = 0;
    for (int i = t; i < V; i += kThreads) top = most(top, key(i));
    top = block_reduce(top, red, most);
    const float m = key_logit((uint32_t)top);
    if (m == -__builtin_inff()) {
        if (t == 0) p.tokens[row] = -1;
        return;
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    const float min_p = p.min_p ? p.min_p[row] : 0.0f;
    const bool greedy = !(temp > 0.0f) || min_p > 1.0f;   // only the first token is kept
    const int top_k = greedy ? 1 : p.top_k ? p.top_k[row] : 0;
    const float T_ = temp > 0.0f ? temp : 1.0f;
    uint32_t cut = 0;
    u64 ties = V;
    if (top_k > 0 && top_k < V) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = cut | (1u << bit);
            u64 c = 0;
            for (int i = t; i < V; i += kThreads) c += key(i) >= trial;
            if (block_reduce(c, red, sum) >= (u64)top_k) cut = trial;
        }
        u64 above = 0;
        for (int i = t; i < V; i += kThreads) above += key(i) > cut;
        ties = top_k - block_reduce(above, red, sum);
    }
    const float top_p = p.top_p ? p.top_p[row] : 1.0f;
    if (!greedy && top_p < 1.0f) {
        // Mass of the top_k tokens, and the lowest key whose predecessors hold less than
        // top_p of it.
        u64 mass = 0, at_cut = 0;
        for (int i = t; i < V; i += kThreads) {
            const uint32_t k = key(i);
            const u64 w = fixed_of(weight_of(key_logit(k), m, T_));
            if (k > cut) mass += w;
            if (k == cut) at_cut += 1;
        }
        mass = block_reduce(mass, red, sum);
        at_cut = block_reduce(at_cut, red, sum);
        mass += min(at_cut, ties) * fixed_of(weight_of(key_logit(cut), m, T_));
        const double limit = (double)top_p * (double)mass;
        auto mass_above = [&](uint32_t x) {
            u64 s = 0;
            for (int i = t; i < V; i += kThreads) {
                const uint32_t k = key(i);
                if (k > x) s += fixed_of(weight_of(key_logit(k), m, T_));
            }
            return block_reduce(s, red, sum);
        };
        uint32_t lo = 0;   // the answer's bits above `bit`; every smaller key fails
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = lo | ((1u << bit) - 1);
            if (!((double)mass_above(trial) < limit)) lo |= 1u << bit;
        }
        const uint32_t pcut = min(lo, (uint32_t)top);
        if (pcut >= cut) {
            const double room = limit - (double)mass_above(pcut);
            const u64 w = fixed_of(weight_of(key_logit(pcut), m, T_));
            // Ties kept: those with fewer than room / w before them.
            u64 r = w ? (u64)fmin(ceil(room / (double)w), 1e9) : (u64)V;
            if (pcut == (uint32_t)top && r < 1) r = 1;
            ties = pcut == cut ? min(ties, r) : r;
            cut = pcut;
        }
    }
    // The race: best score, then lowest index, packed so that the larger wins.
    u64 best = 0, tied = 0;
    for (int base = 0; base < V; base += kThreads) {
        const int i = base + t;
        const uint32_t k = i < V ? key(i) : 0;
        const bool eq = i < V && k == cut;
        const unsigned ballot = __ballot_sync(0xffffffffu, eq);
        __syncthreads();
        if (t % 32 == 0) red[t / 32] = __popc(ballot);
        __syncthreads();
        u64 r = tied + __popc(ballot & ((1u << (t % 32)) - 1));
        for (int j = 0; j < kThreads / 32; ++j) {
            if (j < t / 32) r += red[j];
            tied += red[j];
        }
        if (i >= V || !(k > cut || (eq && r < ties))) continue;
        const float l = key_logit(k);
        if (l == -__builtin_inff()) continue;
        const float w = weight_of(l, m, T_);
        if (w < min_p && !greedy) continue;
        const float score = w / fmaxf(noise[i], 1.17549435e-38f);
        best = most(best, ((u64)__float_as_uint(score) << 32 | (uint32_t)~i));
    }
    best = block_reduce(best, red, most);
    if (t == 0) p.tokens[row] = (uint32_t)~(uint32_t)best;
}

}  // namespace
}  // namespace ctr

extern "C" {

ctr_status ctr_sampler_create(ctr_sampler_t *out, int64_t rows, int64_t vocab, int dtype) {
    if (!out) return CTR_ERR_INVALID_ARG;
    *out = nullptr;
    if (dtype != CTR_F32 && dtype != CTR_BF16 && dtype != CTR_F16) return CTR_ERR_INVALID_ARG;
    if (rows < 0 || vocab < 1) return CTR_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 20) || vocab > ((int64_t)1 << 20)) return CTR_ERR_UNSUPPORTED;
    ctr_sampler_s *pl = new (std::nothrow) ctr_sampler_s();
    if (!pl) return CTR_ERR_INVALID_ARG;
    pl->rows = rows;
    pl->vocab = vocab;
    pl->dtype = dtype;
    *out = pl;
    return CTR_OK;
}

ctr_status ctr_sampler_forward(ctr_sampler_t pl, const void *logits, int64_t logits_stride,
                               const float *noise, int64_t noise_stride,
                               const float *temperature, const int32_t *top_k,
                               const float *top_p, const float *min_p, int64_t *tokens,
                               void *stream) {
    if (!pl) return CTR_ERR_INVALID_ARG;
    if (pl->rows == 0) return CTR_OK;
    if (!logits || !noise || !tokens || logits_stride < pl->vocab || noise_stride < pl->vocab)
        return CTR_ERR_INVALID_ARG;
    auto off = [](const void *q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
    if (off(logits, pl->dtype == CTR_F32 ? 4 : 2) || off(noise, 4) || off(temperature, 4) ||
        off(top_k, 4) || off(top_p, 4) || off(min_p, 4) || off(tokens, 8))
        return CTR_ERR_MISALIGNED;
    ctr::SampleParams p = {logits, noise, logits_stride, noise_stride, temperature, top_p, min_p,
                           top_k, tokens, (int)pl->vocab};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned rows = (unsigned)pl->rows;
    if (pl->dtype == CTR_F32)
        ctr::sample_kernel<float><<<rows, ctr::kThreads, 0, st>>>(p);
    else if (pl->dtype == CTR_BF16)
        ctr::sample_kernel<__nv_bfloat16><<<rows, ctr::kThreads, 0, st>>>(p);
    else
        ctr::sample_kernel<__half><<<rows, ctr::kThreads, 0, st>>>(p);
    ctr::count_launches(1);
    return cudaGetLastError() == cudaSuccess ? CTR_OK : CTR_ERR_CUDA;
}

ctr_status ctr_sampler_describe(ctr_sampler_t pl, char *buf, size_t len) {
    if (!pl || !buf || len == 0) return CTR_ERR_INVALID_ARG;
    static const char *names[] = {"f32", "bf16", "f16"};
    snprintf(buf, len, "sampler %s rows=%lld vocab=%lld", names[pl->dtype], (long long)pl->rows,
             (long long)pl->vocab);
    return CTR_OK;
}

void ctr_sampler_destroy(ctr_sampler_t pl) { delete pl; }

}  // extern "C"
