// attention.cu -- attention of one new token over the paged cache.
#include <algorithm>

#include "attention16.cuh"

namespace ctr {
namespace {

constexpr int kThreads = 128;
constexpr float kNegInf = -__builtin_inff();

__device__ float block_reduce(float v, bool is_max, float *red) {
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = is_max ? fmaxf(v, u) : v + u;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i) v = is_max ? fmaxf(v, red[i]) : v + red[i];
    return v;
}

template <typename T>
__global__ void append_kernel(AttnParams p) {
    const int h = blockIdx.x, b = blockIdx.y;
    int len;
    const int n = tokens_of(p.cache, b, true, &len);
    if (n <= len || len < 0) return;
    const int64_t at = slot_offset(p.cache, b, h, len);
    if (at < 0) return;
    const int64_t src = b * p.kv_stride + (int64_t)h * p.D;
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
        static_cast<T *>(p.k)[at + d] = static_cast<const T *>(p.k_new)[src + d];
        static_cast<T *>(p.v)[at + d] = static_cast<const T *>(p.v_new)[src + d];
    }
}

// One block per (query head, sequence): chunks of 128 slots with the running maximum and sum of
// the softmax; a thread per slot for the scores, a thread per column for the products with V.
template <typename T>
__global__ void attention_kernel(AttnParams p) {
    __shared__ float qs[256], ps[kThreads], red[kThreads / 32];
    __shared__ int64_t offs[kThreads];
    const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x, hk = h / p.G;
    int len;
    const int n = tokens_of(p.cache, b, p.k_new != nullptr, &len);
    const int lo = p.window > 0 && n > p.window ? n - (int)p.window : 0;
    for (int d = t; d < p.D; d += kThreads)
        qs[d] = to_f(static_cast<const T *>(p.q)[b * p.q_stride + (int64_t)h * p.D + d]);
    float m = kNegInf, l = 0.0f, acc[2] = {0.0f, 0.0f};
    float *scores = p.scores ? p.scores + ((int64_t)b * p.Hq + h) * p.score_pitch : nullptr;
    for (int base = lo; base < n; base += kThreads) {
        __syncthreads();
        const int j = base + t;
        float s = kNegInf;
        offs[t] = j < n ? slot_offset(p.cache, b, hk, j) : -1;
        if (offs[t] >= 0) {
            const T *k = static_cast<const T *>(p.k) + offs[t];
            float dot = 0.0f;
            for (int d = 0; d < p.D; ++d) dot = fmaf(qs[d], to_f(k[d]), dot);
            s = dot * p.scale_log2;
        }
        if (scores && j < n) scores[j] = s;
        const float m2 = fmaxf(m, block_reduce(s, true, red));
        const float base_m = m2 == kNegInf ? 0.0f : m2;
        const float e = exp2f(s - base_m), shrink = exp2f(m - base_m);
        ps[t] = e;
        l = l * shrink + block_reduce(e, false, red);
        m = m2;
        for (int i = 0; i < 2; ++i) {
            const int d = t + i * kThreads;
            if (d >= p.D) continue;
            float a = acc[i] * shrink;
            for (int r = 0; r < kThreads && base + r < n; ++r)
                if (offs[r] >= 0) a = fmaf(ps[r], to_f(static_cast<const T *>(p.v)[offs[r] + d]), a);
            acc[i] = a;
        }
    }
    for (int i = 0; i < 2; ++i) {
        const int d = t + i * kThreads;
        if (d < p.D)
            static_cast<T *>(p.out)[((int64_t)b * p.Hq + h) * p.D + d] =
                from_f<T>(l > 0.0f ? acc[i] / l : 0.0f);
    }
    if (scores && t == 0) p.stats[(int64_t)b * p.Hq + h] = make_float2(m, l);
}

__global__ void weights_kernel(AttnParams p, int chunks) {
    const int unit = blockIdx.x / chunks, hk = unit % p.Hkv, b = unit / p.Hkv;
    int len;
    const int n = tokens_of(p.cache, b, p.k_new != nullptr, &len);
    const int lo = p.window > 0 && n > p.window ? n - (int)p.window : 0;
    const int64_t base = ((int64_t)b * p.Hkv + hk) * p.cache.cap, h0 = (int64_t)b * p.Hq + hk * p.G;
    for (int j = blockIdx.x % chunks * blockDim.x + threadIdx.x; j < n; j += chunks * blockDim.x) {
        float w = 0.0f;
        if (j >= lo)
            for (int g = 0; g < p.G; ++g) {
                const float2 st = p.stats[h0 + g];
                if (st.y > 0.0f)
                    w += exp2f(p.scores[(h0 + g) * p.score_pitch + j] - st.x) / st.y;
            }
        p.w_out[base + j] = (p.w_in && j < len ? p.w_in[base + j] : 0.0f) + w;
    }
}

template <typename T, int DP, int NH, int kD>
cudaError_t launch16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    typedef attn16::Shape<DP> Shape;
    static_assert(Shape::kPerSm <= kMaxPerSm && kScoreTile % (16 * Shape::kWarps) == 0, "shape");
    static PerDeviceOnce once;
    const auto kernel = attn16::attention16_kernel<T, DP, NH, kD>;
    cudaError_t e = once.run(current_device(), cudaSuccess, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)attn16::smem_bytes<DP>(DP, 1024));
    });
    if (e != cudaSuccess) return e;
    // Resident blocks: 228 KB an SM, of which a block also takes 1 KB for the system and up to 1 KB
    // of static arrays.  (Large batches' tables of lengths may cost one.)
    const size_t smem = attn16::smem_bytes<DP>(p.D, p.B);
    const int per_sm = std::max(1, std::min(Shape::kPerSm, (int)(228 * 1024 / (smem + 2048))));
    const int grid = pl->num_sms * per_sm;
    count_launches(1);
    e = launch_pdl(kernel, dim3((unsigned)grid), dim3(32 * Shape::kWarps), smem, st, p);
    if (e != cudaSuccess || p.whole_units) return e;
    // Few heads have many parts each: eight warps join one; else two.
    count_launches(1);
    const int64_t heads = (int64_t)p.B * p.Hq;
    if (heads <= 2048)
        return launch_pdl(attn16::join_kernel<T, DP, 8>, dim3((unsigned)heads), dim3(256), 0, st, p, grid);
    return launch_pdl(attn16::join_kernel<T, DP, 2>, dim3((unsigned)((heads + 3) / 4)), dim3(256), 0, st,
                      p, grid);
}

template <typename T, int NH>
cudaError_t launch16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    // Common head sizes have kernels of their own, in which every offset is a constant (1.5 times
    // as fast at 80 columns); the others share one for each 64, 128 or 256.
    switch (p.D) {
    case 64: return launch16<T, 64, NH, 64>(pl, p, st);
    case 80: return launch16<T, 128, NH, 80>(pl, p, st);
    case 96: return launch16<T, 128, NH, 96>(pl, p, st);
    case 128: return launch16<T, 128, NH, 128>(pl, p, st);
    case 256: return launch16<T, 256, NH, 256>(pl, p, st);
    }
    return p.D < 64    ? launch16<T, 64, NH, 0>(pl, p, st)
           : p.D < 128 ? launch16<T, 128, NH, 0>(pl, p, st)
                       : launch16<T, 256, NH, 0>(pl, p, st);
}

template <typename T>
cudaError_t launch16(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    return p.G <= 8 ? launch16<T, 1>(pl, p, st) : launch16<T, 2>(pl, p, st);
}

template <typename T>
cudaError_t launch(const AttnParams &p, cudaStream_t st) {
    if (p.k_new) {
        append_kernel<T><<<dim3(p.Hkv, p.B), kThreads, 0, st>>>(p);
        count_launches(1);
    }
    attention_kernel<T><<<dim3(p.Hq, p.B), kThreads, 0, st>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const ctr_attn_s *pl, const AttnParams &p, cudaStream_t st) {
    cudaError_t e = pl->dtype == CTR_F32    ? launch<float>(p, st)
                    : pl->dtype == CTR_BF16 ? launch16<__nv_bfloat16>(pl, p, st)
                                            : launch16<__half>(pl, p, st);
    if (e != cudaSuccess || !p.w_out) return e;
    const int chunks = std::min((p.cache.cap + 1023) / 1024, 64);
    weights_kernel<<<(unsigned)(p.B * p.Hkv) * chunks, 256, 0, st>>>(p, chunks);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ctr
