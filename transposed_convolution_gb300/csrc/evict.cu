// evict.cu -- eviction from the paged cache by accumulated attention weight.
#include <algorithm>

#include "decode_device.cuh"

namespace ctr {
namespace {

constexpr int kSelectThreads = 512;

// Order-preserving key: larger weight, larger key; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ int block_sum(int v, int *red) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kSelectThreads / 32; ++i) v += red[i];
    return v;
}

// One block per (sequence, KV head): the smallest key that stays, found bit by bit, then the
// kept slots in order by a scan over the slots.
__global__ void select_kernel(EvictParams p) {
    __shared__ int red[kSelectThreads / 32];
    const int unit = blockIdx.x, b = unit / p.Hkv, t = threadIdx.x;
    const int len = p.cache.lens[b];
    int n = len < 0 ? 0 : len;
    if (n > p.cache.cap) {
        n = p.cache.cap;
        if (t == 0) atomicOr(p.cache.status, kStatusBadLength);
    }
    const int keep = min(n, p.budget);
    const float *w = p.w + (int64_t)unit * p.cache.cap;
    const int s0 = min(p.sinks, n), r0 = max(s0, n - p.recent);   // the others: s0 <= j < r0
    const int want = keep - s0 - (n - r0);                        // of the others
    uint32_t cut = 0;      // the want-th largest key
    int ties = 0;          // how many of the slots with key == cut stay
    if (want > 0 && want < r0 - s0) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = cut | (1u << bit);
            int c = 0;
            for (int j = s0 + t; j < r0; j += kSelectThreads) c += weight_key(w[j]) >= trial;
            if (block_sum(c, red) >= want) cut = trial;
        }
        int above = 0;
        for (int j = s0 + t; j < r0; j += kSelectThreads) above += weight_key(w[j]) > cut;
        ties = want - block_sum(above, red);
    }
    const bool all = want >= r0 - s0;
    int32_t *slots = p.slots + (int64_t)unit * p.budget;
    int done = 0, tied = 0;      // kept slots and ties before this round
    for (int base = 0; base < n; base += kSelectThreads) {
        const int j = base + t;
        bool eq = false, on = false;
        if (j < n) {
            on = j < s0 || j >= r0 || all;
            if (!on && want > 0) {
                const uint32_t k = weight_key(w[j]);
                on = k > cut;
                eq = k == cut;
            }
        }
        // Ranks inside the round: ties first, then the kept.
        const unsigned be = __ballot_sync(0xffffffffu, eq), before = (1u << (t % 32)) - 1;
        __syncthreads();
        if (t % 32 == 0) red[t / 32] = __popc(be);
        __syncthreads();
        int r = tied + __popc(be & before);
        for (int i = 0; i < t / 32; ++i) r += red[i];
        for (int i = 0; i < kSelectThreads / 32; ++i) tied += red[i];
        if (eq && r < ties) on = true;
        const unsigned bo = __ballot_sync(0xffffffffu, on);
        __syncthreads();
        if (t % 32 == 0) red[t / 32] = __popc(bo);
        __syncthreads();
        r = done + __popc(bo & before);
        for (int i = 0; i < t / 32; ++i) r += red[i];
        for (int i = 0; i < kSelectThreads / 32; ++i) done += red[i];
        if (on) slots[r] = j;
    }
    for (int i = keep + t; i < p.budget; i += kSelectThreads) slots[i] = -1;
    if (unit % p.Hkv == 0 && t == 0) p.lens_out[b] = len < 0 ? len : keep;
}

// One warp per kept row: K, V and the weight to the destination slot.
__global__ void copy_kernel(EvictParams p, int chunks) {
    const int unit = blockIdx.x / chunks, b = unit / p.Hkv, h = unit % p.Hkv;
    const int warps = blockDim.x / 32;
    for (int i = blockIdx.x % chunks * warps + threadIdx.x / 32; i < p.budget; i += chunks * warps) {
        const int j = p.slots[(int64_t)unit * p.budget + i];
        if (j < 0) break;
        const int64_t src = slot_offset(p.cache, b, h, j);
        const int pg = p.dst_tables[b * p.dst_pitch + i / p.cache.page];
        if ((unsigned)pg >= (unsigned)p.cache.num_pages) {
            atomicOr(p.cache.status, kStatusBadPage);
            continue;
        }
        const int64_t dst = pg * p.cache.page_stride + h * p.cache.head_stride +
                            (i % p.cache.page) * p.cache.row_stride;
        if (src >= 0) {
            for (int c = threadIdx.x % 32; c < p.row_bytes / 16; c += 32) {
                const uint4 k = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.k) + src * p.esize)[c];
                const uint4 v = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.v) + src * p.esize)[c];
                reinterpret_cast<uint4 *>(static_cast<char *>(p.k) + dst * p.esize)[c] = k;
                reinterpret_cast<uint4 *>(static_cast<char *>(p.v) + dst * p.esize)[c] = v;
            }
        }
        if (p.w_out && threadIdx.x % 32 == 0)
            p.w_out[unit * p.w_pitch + i] = p.w[(int64_t)unit * p.cache.cap + j];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t st) {
    const int units = p.B * p.Hkv;
    select_kernel<<<units, kSelectThreads, 0, st>>>(p);
    const int chunks = std::min((p.budget + 31) / 32, 1024);
    copy_kernel<<<(unsigned)units * chunks, 256, 0, st>>>(p, chunks);
    count_launches(2);
    return cudaGetLastError();
}

}  // namespace ctr
