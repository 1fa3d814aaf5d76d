// evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Two kernels.  The first reads each (sequence, KV head)'s weights once, as order-preserving keys
// in shared memory where they fit, finds the lowest key that stays by three histograms (11, 11
// and 10 bits), and lists the kept slots in order: counts by warp, their sum, and the list, which
// takes a ballot for each 32 slots.  Few long sequences are spread over clusters of blocks, which add up
// their histograms (32767 slots of 16 heads: 24 us in 16 blocks, 16 in 64).  The second copies the
// listed rows; it moves 4 D elements a row and is bound by the cache's memory, so its blocks are many
// and small, each with the row addresses of 64 rows in shared memory and two 16-byte loads of K and
// V under way for each thread at a time.  It is launched while the first still runs, and waits for
// its end.
#include <algorithm>
#include <cooperative_groups.h>

#include "decode_device.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace ctr {
namespace {

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kStageKeys = 40 * 1024;      // most keys a block keeps in shared memory (160 KB)
// Clusters of eight such blocks leave too few free SMs a GPC for a second one everywhere.
constexpr int kMaxCluster = 4, kPartSlots = 4096;
constexpr int kCopyThreads = 256, kCopyRows = 64;

// Order-preserving key: larger weight, larger key; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of two counts by warp, and their totals.  Not inlined, so that lanes meet
// at one copy of its shuffles.
__device__ __noinline__ void scan_warps(int (&a)[kSelectWarps], int (&b)[kSelectWarps]) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int x = a[lane], y = b[lane];
        int xi = x, yi = y;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, xi, o), v = __shfl_up_sync(0xffffffffu, yi, o);
            if (lane >= o) {
                xi += u;
                yi += v;
            }
        }
        a[lane] = xi - x;
        b[lane] = yi - y;
    }
    __syncthreads();
}

struct Boundary {
    int bin, before, inside;
};

// The bin of the histogram, from the top one down, in which the count reaches `target`.
__device__ __noinline__ void find_bin(const int (&hist)[kBins], int target, int (&warp_a)[kSelectWarps],
                                      Boundary *found) {
    constexpr int kEach = kBins / kSelectThreads;
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    int c[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        c[i] = hist[kBins - 1 - (t * kEach + i)];
        sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_a[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int i = 0; i < warp; ++i) before += warp_a[i];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (before < target && target <= before + c[i])
            *found = Boundary{kBins - 1 - (t * kEach + i), before, c[i]};
        before += c[i];
    }
    __syncthreads();
}

// One cluster for each (sequence, KV head), each block a run of `part` slots.
template <bool kStaged>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(EvictParams p, int part) {
    extern __shared__ __align__(16) unsigned char staged[];
    // A histogram a round, so that a block may go on while others still read its last one.
    __shared__ int hists[3][kBins], sums[kBins], warp_a[kSelectWarps], warp_b[kSelectWarps];
    __shared__ int counts[kMaxCluster][2];
    __shared__ Boundary found;
    uint32_t *const keys = reinterpret_cast<uint32_t *>(staged);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / C, b = unit / p.Hkv, t = threadIdx.x, lane = t % 32, warp = t / 32;
    // No block touches another's shared memory before all of the cluster have started: there may be
    // nothing to choose, and the first access is then the counts'.
    if (C > 1) ptx::cluster_arrive_relaxed();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int len = p.cache.lens[b];
    int n = max(len, 0);
    if (n > p.cache.cap) {
        n = p.cache.cap;
        if (t == 0) atomicOr(p.cache.status, kStatusBadLength);
    }
    if (C > 1) ptx::cluster_wait();
    const int first = min(rank * part, n), last = min(first + part, n);     // this block's slots
    const int keep = min(n, p.budget);
    const float *const w = p.w + (int64_t)unit * p.cache.cap;
    const int s0 = min(p.sinks, n), r0 = max(s0, n - p.recent);   // the others: s0 <= j < r0
    const int want = keep - s0 - (n - r0);                        // of the others
    const bool all = want >= r0 - s0;
    auto key_at = [&](int j) { return kStaged ? keys[j - first] : weight_key(w[j]); };

    // The lowest key that stays, by histograms of its bits from the top.
    uint32_t cut = 0;
    int ties = 0;          // how many of the others with key == cut stay
    if (want > 0 && !all) {
        int target = want, above = 32;      // bits of the keys not yet decided
        const int from = max(first, s0), to = min(last, r0);
        for (int round = 0; round < 3; ++round) {
            int (&hist)[kBins] = hists[round];
            const int bits = round < 2 ? 11 : 10, shift = above - bits;
            for (int i = t; i < kBins; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int j = from + t; j < to; j += kSelectThreads) {
                uint32_t k;
                if (round == 0) {
                    k = weight_key(w[j]);
                    if (kStaged) keys[j - first] = k;
                } else {
                    k = key_at(j);
                }
                if (round == 0 || k >> above == cut >> above)
                    atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1);
            }
            if (C > 1) {
                cluster.sync();
                for (int i = t; i < kBins; i += kSelectThreads) {
                    int sum = 0;
                    for (int c = 0; c < C; ++c) sum += cluster.map_shared_rank(&hist[0], c)[i];
                    sums[i] = sum;
                }
            }
            __syncthreads();
            find_bin(C > 1 ? sums : hist, target, warp_a, &found);
            cut |= (uint32_t)found.bin << shift;
            target -= found.before;
            above = shift;
            // The whole bin stays: nothing below is to be decided.
            if (found.inside == target) {
                target = 0x7fffffff;
                break;
            }
            __syncthreads();
        }
        ties = target;
    }
    const bool whole_bin = ties == 0x7fffffff;     // every key >= cut stays
    __syncthreads();

    // The list: each warp takes a run of the block's slots.
    const int run = ((last - first + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int from = min(first + warp * run, last), to = min(from + run, last);
    auto decide = [&](int j, bool *on, bool *eq) {
        *on = *eq = false;
        if (j >= to) return;
        *on = j < s0 || j >= r0 || all;
        if (!*on && want > 0) {
            const uint32_t k = key_at(j);
            *on = whole_bin ? k >= cut : k > cut;
            *eq = !whole_bin && k == cut;
        }
    };
    int sure = 0, equal = 0;
    for (int base = from; base < to; base += 32) {
        bool on, eq;
        decide(base + lane, &on, &eq);
        sure += __popc(__ballot_sync(0xffffffffu, on));
        equal += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        warp_a[warp] = sure;
        warp_b[warp] = equal;
    }
    scan_warps(warp_a, warp_b);
    int sure_before = warp_a[warp], tie = warp_b[warp];
    if (C > 1) {
        // The last warp has the block's totals: to every block.
        if (warp == kSelectWarps - 1 && lane < C) {
            int (*to_counts)[2] = cluster.map_shared_rank(&counts[0], lane);
            to_counts[rank][0] = sure_before + sure;
            to_counts[rank][1] = tie + equal;
        }
        cluster.sync();
        for (int c = 0; c < rank; ++c) {
            sure_before += counts[c][0];
            tie += counts[c][1];
        }
    }
    int at = sure_before + min(tie, ties);
    int32_t *const slots = p.slots + (int64_t)unit * p.budget;
    const unsigned below = (1u << lane) - 1;
    for (int base = from; base < to; base += 32) {
        bool on, eq;
        decide(base + lane, &on, &eq);
        const unsigned be = __ballot_sync(0xffffffffu, eq);
        if (eq && tie + __popc(be & below) < ties) on = true;
        tie += __popc(be);
        const unsigned bo = __ballot_sync(0xffffffffu, on);
        if (on) slots[at + __popc(bo & below)] = base + lane;
        at += __popc(bo);
    }
    if (rank == 0) {
        for (int i = keep + t; i < p.budget; i += kSelectThreads) slots[i] = -1;
        if (unit % p.Hkv == 0 && t == 0) p.lens_out[b] = len < 0 ? len : keep;
    }
}

// kCopyRows kept rows of one (sequence, KV head) a block: K, V and weights.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(EvictParams p, int blocks_a_unit) {
    __shared__ int64_t from[kCopyRows], to[kCopyRows];     // 16-byte chunks; -1: not to be copied
    const int unit = blockIdx.x / blocks_a_unit, b = unit / p.Hkv, h = unit % p.Hkv;
    const int i0 = blockIdx.x % blocks_a_unit * kCopyRows, t = threadIdx.x;
    ptx::griddep_wait();
    if (t < kCopyRows) {
        const int i = i0 + t, j = i < p.budget ? p.slots[(int64_t)unit * p.budget + i] : -1;
        int64_t src = -1, dst = -1;
        if (j >= 0) {
            src = slot_offset(p.cache, b, h, j);
            const int pg = p.dst_tables[b * p.dst_pitch + i / p.cache.page];
            if ((unsigned)pg >= (unsigned)p.cache.num_pages) {
                atomicOr(p.cache.status, kStatusBadPage);
                src = -1;
            } else {
                dst = pg * p.cache.page_stride + h * p.cache.head_stride +
                      (i % p.cache.page) * p.cache.row_stride;
            }
            if (p.w_out) p.w_out[unit * p.w_pitch + i] = p.w[(int64_t)unit * p.cache.cap + j];
        }
        from[t] = src < 0 ? -1 : src * p.esize / 16;
        to[t] = dst * p.esize / 16;
    }
    __syncthreads();
    const int chunks = p.row_bytes / 16, total = kCopyRows * chunks;
    const uint4 *const k = static_cast<const uint4 *>(p.k), *const v = static_cast<const uint4 *>(p.v);
    uint4 *const ko = static_cast<uint4 *>(p.k), *const vo = static_cast<uint4 *>(p.v);
    for (int x0 = t; x0 < total; x0 += 2 * kCopyThreads) {
        uint4 a[2], c[2];
        int64_t at[2];
        // Past the end the last chunk is read again, for nothing, as are chunks of no row.
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = min(x0 + u * kCopyThreads, total - 1), r = x / chunks, e = x - r * chunks;
            const int64_t f = from[r] < 0 ? 0 : from[r];
            at[u] = from[r] < 0 || x0 + u * kCopyThreads >= total ? -1 : to[r] + e;
            a[u] = k[f + e];
            c[u] = v[f + e];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (at[u] >= 0) {
                ko[at[u]] = a[u];
                vo[at[u]] = c[u];
            }
    }
}

template <bool kStaged>
cudaError_t launch_select(const EvictParams &p, int units, int cluster, int part, cudaStream_t st) {
    static PerDeviceOnce once;
    const cudaError_t e = once.run(current_device(), cudaSuccess, [] {
        return cudaFuncSetAttribute(select_kernel<kStaged>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kStaged ? kStageKeys * (int)sizeof(uint32_t) : 0);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = kStaged ? (size_t)part * sizeof(uint32_t) : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<kStaged>, p, part);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t st) {
    const int units = p.B * p.Hkv;
    // Blocks a unit: two an SM for few units, but kPartSlots slots each at least.
    int cluster = 1;
    while (cluster < kMaxCluster && (int64_t)units * cluster <= p.num_sms &&
           p.cache.cap >= 2 * cluster * kPartSlots)
        cluster *= 2;
    const int part = ((p.cache.cap + cluster - 1) / cluster + 31) / 32 * 32;
    cudaError_t e = part <= kStageKeys ? launch_select<true>(p, units, cluster, part, st)
                                       : launch_select<false>(p, units, cluster, part, st);
    if (e != cudaSuccess) return e;
    const int blocks = (int)((std::min<int64_t>(p.budget, p.cache.cap) + kCopyRows - 1) / kCopyRows);
    count_launches(2);
    return launch_pdl(copy_kernel, dim3((unsigned)units * blocks), dim3(kCopyThreads), 0, st, p, blocks);
}

}  // namespace ctr
