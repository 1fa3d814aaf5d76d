// sampler.cu -- sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// Every filter keeps a prefix of the order (logit descending, index ascending), so the kept set
// is a lowest key, and how many of the tokens with that key stay.  The logits are read once, which
// bounds the operator: V elements of 2 or 4 bytes a row, and the random numbers of the kept
// tokens only.  25 million of them take the CUDA cores longer than the memory (23 instructions a logit
// in all with top-p and min-p: 33 us, 7.5 of them the memory's), so the work on each is kept to half a packed
// maximum, and for top-p a conversion, a scaled difference and an exponential while the memory is busy.
// A row's block (or cluster of blocks)
//   1. reads its part into shared memory, where it fits, and takes the maximum and the mass;
//   2. lists the tokens within 2^-kListBits of the maximum (or min_p of it: nothing below is kept
//      then) at the cluster's first block; the others wait;
//   3. finds the cuts among the listed tokens, by a histogram of their distance to the maximum
//      and, inside the bin that a cut falls into, histograms of their keys;
//   4. races the kept ones: best w / noise, ties to the lowest index.
// Where the list cannot hold the cuts (flat logits without min_p, or too many tokens near the maximum)
// all blocks do 3 and 4 together, each on its part: every histogram is the sum of theirs, and each
// races its own.  16 rows of 200000 fp32 logits, top-p 0.95 at temperature 1.3 (a fifth of the tokens
// stays): 111 us from memory and 102 partly from L2, with 25000 logits a block gone over eight times; by
// one block of the row alone 420.
//
// Sums: a thread's masses are added in fp32 in a fixed order, everything beyond as integers in units of
// 2^-35, and the list's order matters to nothing: equal inputs give equal tokens.  A bin's mass is
// three 32-bit counters of twelve bits' worth each, because 64-bit additions in shared memory are
// loops of compare-and-swap (1.8 to 100 times as slow, by how often they meet).
#include <algorithm>
#include <cooperative_groups.h>
#include <cstdio>
#include <new>

#include "decode_device.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

struct ctr_sampler_s {
    int64_t rows, vocab;
    int dtype, num_sms;
};

namespace ctr {
namespace {

typedef unsigned long long u64;
constexpr float kNegInf = -__builtin_inff();
constexpr int kBins = 1024;
constexpr int kListMax = 3000;
constexpr float kListBits = 12.0f;    // tokens within 2^-12 of the maximum are listed
constexpr int kMaxCluster = 8;
// Most logits a block keeps in shared memory, two blocks an SM, and one.
constexpr int kStageBytes = 58 * 1024, kStageBytesAlone = 160 * 1024;

struct SampleParams {
    const void *logits;
    const float *noise;
    int64_t logits_stride, noise_stride;
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *tokens;
    int vocab, chunk;        // elements of a row, and of a block's part (a multiple of 16)
};

// Order-preserving key of a logit (NaN as -inf, -0 as +0) and back.
__device__ __forceinline__ uint32_t logit_key(float l) {
    const uint32_t u = __float_as_uint(fmaxf(l, kNegInf) + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// w_i = exp((l - m) / T), 1 at the maximum (also when it is infinite).
__device__ __forceinline__ float weight_of(float l, float m, float T) {
    return l == m ? 1.0f : expf((l - m) / T);
}
// Masses are sums of weights (at most 1, up to 2^20 of them) in units of 2^-35.
__device__ __forceinline__ u64 fixed_of(float w) { return __float2ull_rn(w * 34359738368.0f); }
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The best score so far and its index; equal scores go to the lower one.
struct Best {
    float score = -1.0f;
    int index = 0;
    __device__ __forceinline__ void offer(float v, int i) {
        if (v > score || (v == score && i < index)) {
            score = v;
            index = i;
        }
    }
    // Larger is better; 0 for none.
    __device__ __forceinline__ u64 packed() const {
        return score < 0.0f ? 0 : (u64)__float_as_uint(score) << 32 | (uint32_t)~index;
    }
};

// Weights in powers of two, for masses: a relative error of 2^-22 moves a cut by less than
// rounding the logits does.
struct Scale {
    float m, c;              // the maximum, and log2(e) / T
    // log2 of the weight; 0 at the maximum also where that is infinite, or the scale.
    __device__ __forceinline__ float below(float l) const { return l == m ? 0.0f : (l - m) * c; }
    __device__ __forceinline__ float mass(float l) const { return pow2(fmaxf(below(l), -200.0f)); }
};

// The kept prefix: keys above `low`, and of those equal to it the `ties` with the lowest indices.
struct Cut {
    uint32_t low;
    uint32_t ties;           // 0xffffffff: all
};

struct Listed {
    uint32_t key, index;
};
constexpr int kLocalMax = 2048;      // tokens listed by one block
constexpr uint32_t kSpoilt = 1u << 24;

// The blocks that search together: one alone, or all of a cluster.
struct Alone {
    static constexpr int count = 1;
    __device__ __forceinline__ void sync() const { __syncthreads(); }
    template <typename S> __device__ __forceinline__ const S &of(S &s, int) const { return s; }
};
struct Together {
    int count;
    __device__ __forceinline__ void sync() const { cg::this_cluster().sync(); }
    template <typename S> __device__ __forceinline__ const S &of(S &s, int r) const {
        return *cg::this_cluster().map_shared_rank(&s, r);
    }
};

// (A multiple of 16 bytes: the staged logits lie behind it.)
template <int kThreads> struct __align__(16) Shared {
    u64 red[kThreads / 32], red2[kThreads / 32];
    union {
        // A histogram: counts, masses (twelve bits each, the lowest first), lowest and highest keys.
        struct {
            uint32_t count[kBins], mass[3][kBins], low[kBins], high[kBins];
        };
        Listed local[kLocalMax];         // before that, this block's tokens for the list
    };
    // What a boundary search found: its bin and the counts and masses before and in it.
    uint32_t bin, before, inside;
    u64 mass_before, mass_inside, mass_sum, target;
    uint32_t rest, rest_low, rest_high;  // the last bin's count and keys
    u64 rest_mass;                       // and mass
    int locals;
    // Written by the cluster's blocks: the maxima at every block, the others at the first.
    uint32_t tops[kMaxCluster];
    u64 bests[kMaxCluster];
    u64 totals[kMaxCluster];             // mass of each part
    uint32_t listed;                     // tokens for the list, and kSpoilt for each block with too many
    int wide;                            // the list does not do: all blocks go on
    Listed list[kListMax];
};

// The largest (or the sum) of the block's values.  Not inlined: behind a loop that lanes leave at
// different times, nvcc 13.0.88 otherwise copies the shuffles into both ways out of it, and lanes
// that meet at different copies do not see one another.
template <int kThreads, bool kSum> __device__ __noinline__ u64 block_reduce(u64 v, u64 *red) {
    auto f = [](u64 a, u64 b) { return kSum ? a + b : a > b ? a : b; };
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v = f(v, red[i]);
    return v;
}
template <int kThreads> __device__ __forceinline__ u64 block_max(u64 v, u64 *red) {
    return block_reduce<kThreads, false>(v, red);
}
template <int kThreads> __device__ __forceinline__ u64 block_sum(u64 v, u64 *red) {
    return block_reduce<kThreads, true>(v, red);
}

// 16 bytes' elements as fp32, and the largest of them (NaN only if all are).
__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4], float) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ __half2 pair_of(uint32_t u, __half) {
    return __halves2half2(__ushort_as_half((unsigned short)u), __ushort_as_half((unsigned short)(u >> 16)));
}
__device__ __forceinline__ __nv_bfloat162 pair_of(uint32_t u, __nv_bfloat16) {
    return __halves2bfloat162(__ushort_as_bfloat16((unsigned short)u),
                              __ushort_as_bfloat16((unsigned short)(u >> 16)));
}
__device__ __forceinline__ float2 floats_of(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ float2 floats_of(__nv_bfloat162 v) { return __bfloat1622float2(v); }
template <typename T> __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8], T tag) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = floats_of(pair_of(w[i], tag));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ float max_of(const uint4 &u, float) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                 fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <typename T> __device__ __forceinline__ float max_of(const uint4 &u, T tag) {
    const float2 f = floats_of(__hmax2(__hmax2(pair_of(u.x, tag), pair_of(u.y, tag)),
                                       __hmax2(pair_of(u.z, tag), pair_of(u.w, tag))));
    return fmaxf(f.x, f.y);
}

// Bits of -inf.
__device__ __forceinline__ uint32_t neg_inf_bits(float) { return 0xff800000u; }
__device__ __forceinline__ uint32_t neg_inf_bits(__half) { return 0xfc00u; }
__device__ __forceinline__ uint32_t neg_inf_bits(__nv_bfloat16) { return 0xff80u; }

// A block's part of a row, 16 bytes at a time from the 16-byte boundary `skew` elements before it;
// what a vector holds beside the part's elements reads as -inf, which no filter keeps.
template <typename T> struct Part {
    const T *at;             // the boundary
    int skew, count;
    int base;                // index of the first element
    static constexpr int kVec = 16 / sizeof(T);
    __device__ __forceinline__ int vecs() const { return (skew + count + kVec - 1) / kVec; }
    __device__ __forceinline__ int index(int v) const { return base + v * kVec - skew; }
    __device__ __forceinline__ uint4 load(int v) const {
        const int first = v * kVec - skew;
        if (first >= 0 && first + kVec <= count) return __ldg(reinterpret_cast<const uint4 *>(at) + v);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sizeof(T) == 4) {
                w[i] = (unsigned)(first + i) < (unsigned)count
                           ? __ldg(reinterpret_cast<const uint32_t *>(at) + v * kVec + i) : neg_inf_bits(T());
            } else {
                w[i] = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = 2 * i + h;
                    const uint32_t x = (unsigned)(first + e) < (unsigned)count
                                           ? (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(at) + v * kVec + e)
                                           : neg_inf_bits(T());
                    w[i] |= x << (16 * h);
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int kThreads> __device__ __forceinline__ void clear_bins(Shared<kThreads> &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads)
    {
        s.count[i] = s.mass[0][i] = s.mass[1][i] = s.mass[2][i] = s.high[i] = 0;
        s.low[i] = 0xffffffffu;
    }
}
// One element to a bin; 2^20 of them overflow no counter.
template <int kThreads> __device__ __forceinline__ void add_to_bin(Shared<kThreads> &s, int bin, u64 w) {
    atomicAdd(&s.count[bin], 1u);
    if (w == 0) return;
    atomicAdd(&s.mass[0][bin], (uint32_t)w & 0xfffu);
    atomicAdd(&s.mass[1][bin], (uint32_t)(w >> 12) & 0xfffu);
    atomicAdd(&s.mass[2][bin], (uint32_t)(w >> 24));
}

// Finds the boundary bin of the peers' histograms together: the first whose counts (or masses)
// bring the sum to `target`, or to that share of the total mass, and the total mass.  Without one (the
// total is less) it is the last bin.  Called by all threads, whose histograms are complete.
template <int kThreads, typename Peers>
__device__ __noinline__ void find_bin(Shared<kThreads> &s, Peers peers, bool by_mass, bool weigh, u64 target,
                                      float share) {
    constexpr int kEach = kBins / kThreads;
    static_assert(kBins % kThreads == 0, "bins");
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    u64 c[kEach] = {}, m[kEach] = {}, cs = 0, ms = 0;
#pragma unroll 4
    for (int r = 0; r < peers.count; ++r) {
        const Shared<kThreads> &o = peers.of(s, r);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            c[i] += o.count[t * kEach + i];
            if (weigh)
                m[i] += (u64)o.mass[0][t * kEach + i] + ((u64)o.mass[1][t * kEach + i] << 12) +
                        ((u64)o.mass[2][t * kEach + i] << 24);
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        cs += c[i];
        ms += m[i];
    }
    __syncwarp();
    u64 ci = cs, mi = ms;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const u64 a = __shfl_up_sync(0xffffffffu, ci, o), b = __shfl_up_sync(0xffffffffu, mi, o);
        if (lane >= o) {
            ci += a;
            mi += b;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.red[warp] = ci;
        s.red2[warp] = mi;
    }
    if (t == 0) s.bin = kBins - 1;
    __syncthreads();
    u64 cb = ci - cs, mb = mi - ms;
    for (int i = 0; i < warp; ++i) {
        cb += s.red[i];
        mb += s.red2[i];
    }
    if (share > 0.0f) {
        u64 all = 0;
        for (int i = 0; i < kThreads / 32; ++i) all += s.red2[i];
        target = max((u64)1, (u64)ceil((double)share * (double)all));
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const u64 b = by_mass ? mb : cb, in = by_mass ? m[i] : c[i];
        if (b < target && target <= b + in) {
            s.bin = t * kEach + i;
            s.before = (uint32_t)cb;
            s.inside = (uint32_t)c[i];
            s.mass_before = mb;
            s.mass_inside = m[i];
        }
        cb += c[i];
        mb += m[i];
    }
    if (t == kThreads - 1) {
        s.mass_sum = mb;
        s.target = target;
    }
    __syncthreads();
}

// The cut among `inside` elements of one key, of mass `in` together: the first so many of them.
__device__ __forceinline__ Cut cut_of_one_key(uint32_t key, uint32_t inside, bool by_mass, u64 target, u64 before,
                                              u64 above, u64 in, u64 *mass) {
    const u64 w = in / inside;
    u64 r = by_mass ? (w ? (target - above + w - 1) / w : inside) : target - before;
    r = max((u64)1, min(r, (u64)inside));
    *mass = above + r * w;
    return Cut{key, r == inside ? 0xffffffffu : (uint32_t)r};
}

// Histograms of keys in [lo, hi], each of the bin of the last one that the boundary falls into, until
// that holds one key, one element, or is kept whole.  each(f) calls f(key, weight()) of every
// element that this block has; count0 and mass0 are of the elements above hi.
template <int kThreads, typename Peers, typename Each>
__device__ Cut cut_by_keys(Shared<kThreads> &s, Peers peers, uint32_t lo, uint32_t hi, bool by_mass, bool weigh,
                           u64 target, u64 count0, u64 mass0, u64 *mass, Each each) {
    for (;;) {
        const int shift = max(0, 32 - __clz(hi - lo) - 10);
        clear_bins(s);
        __syncthreads();
        each([&](uint32_t key, auto weight) {
            if (key >= lo && key <= hi) add_to_bin(s, (int)((hi - key) >> shift), weight());
        });
        peers.sync();
        find_bin<kThreads>(s, peers, by_mass, weigh, target - (by_mass ? mass0 : count0), 0.0f);
        const uint32_t bin = s.bin, inside = s.inside;
        const u64 before = count0 + s.before, above = mass0 + s.mass_before, in = s.mass_inside;
        peers.sync();
        const uint32_t top = hi - (bin << shift);
        const uint32_t low = top - lo < (1u << shift) ? lo : top - ((1u << shift) - 1);
        if (inside == 1 || (!by_mass && before + inside == target)) {
            *mass = above + in;
            return Cut{low, 0xffffffffu};
        }
        if (shift == 0) return cut_of_one_key(low, inside, by_mass, target, before, above, in, mass);
        count0 = before;
        mass0 = above;
        hi = top;
        lo = low;
    }
}

// The cut at which the count (or, by_mass, the mass) of the prefix reaches `target`, or `share` of the
// total mass, over the elements that each(key, f) passes to f(logit) in the peers' blocks (it may leave
// out those below the key), without those whose keys are below `floor_key`; *found is false where they
// have less mass than that.  *mass is the mass of the prefix, where `weigh`.  First a histogram of the
// distance to the maximum, in kBins - 1 steps over `range` powers of two and one for the rest.
template <int kThreads, typename Peers, typename Each>
__device__ Cut find_cut(Shared<kThreads> &s, Peers peers, const Scale &scale, float range, bool by_mass, bool weigh,
                        u64 target, float share, uint32_t floor_key, u64 *mass, bool *found, Each each) {
    const float steps = (kBins - 1) / range;
    auto bin_of = [&](float l) { return min(kBins - 1, (int)(-scale.below(l) * steps)); };
    auto weight = [&](float l) { return weigh ? fixed_of(scale.mass(l)) : 0; };
    clear_bins(s);
    if (threadIdx.x == 0) {
        s.rest = s.rest_high = 0;
        s.rest_low = 0xffffffffu;
        s.rest_mass = 0;
    }
    __syncthreads();
    uint32_t rest = 0, rest_low = 0xffffffffu, rest_high = 0;
    u64 rest_mass = 0;
    each(max(floor_key, logit_key(kNegInf)), [&](float l) {
        const uint32_t key = logit_key(l);
        if (key < floor_key) return;
        const int bin = bin_of(l);
        const u64 w = weight(l);
        if (bin == kBins - 1) {
            ++rest;
            rest_mass += w;
            rest_low = min(rest_low, key);
            rest_high = max(rest_high, key);
        } else {
            add_to_bin(s, bin, w);
            atomicMin(&s.low[bin], key);
            atomicMax(&s.high[bin], key);
        }
    });
    // The last bin's elements are counted by thread: there may be nearly all of them.
    if (rest) {
        atomicAdd(&s.rest, rest);
        atomicAdd(&s.rest_mass, rest_mass);
        atomicMin(&s.rest_low, rest_low);
        atomicMax(&s.rest_high, rest_high);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s.count[kBins - 1] = s.rest;
        s.mass[0][kBins - 1] = (uint32_t)s.rest_mass & 0xfffu;
        s.mass[1][kBins - 1] = (uint32_t)(s.rest_mass >> 12) & 0xfffu;
        s.mass[2][kBins - 1] = (uint32_t)(s.rest_mass >> 24);
        s.low[kBins - 1] = s.rest_low;
        s.high[kBins - 1] = s.rest_high;
    }
    peers.sync();
    find_bin<kThreads>(s, peers, by_mass, weigh, target, share);
    const int bin = s.bin;
    uint32_t low = 0xffffffffu, high = 0;
#pragma unroll 4
    for (int r = 0; r < peers.count; ++r) {
        low = min(low, peers.of(s, r).low[bin]);
        high = max(high, peers.of(s, r).high[bin]);
    }
    const uint32_t inside = s.inside;
    const u64 before = s.before, above = s.mass_before, in = s.mass_inside;
    target = s.target;
    *found = !by_mass || target <= s.mass_sum;
    peers.sync();
    if (!*found) return Cut{0, 0xffffffffu};
    if (inside == 1 || (!by_mass && before + inside == target)) {
        *mass = above + in;
        return Cut{low, 0xffffffffu};
    }
    if (low == high) return cut_of_one_key(low, inside, by_mass, target, before, above, in, mass);
    return cut_by_keys<kThreads>(s, peers, low, high, by_mass, weigh, target, before, above, mass, [&](auto f) {
        each(low, [&](float l) { f(logit_key(l), [&]() { return weight(l); }); });
    });
}

// What is asked of a row whose maximum is m: by_min holds by itself.
struct Query {
    const float *noise;
    float m, c, T, min_p, top_p;
    int asked, V;
    bool by_k, by_p, to_min;
    // N tokens race, those whose `keep` is set.  All numbers are asked for before the first is used
    // (token 0's for those that are out: loads behind a condition would wait for one another).
    template <int N>
    __device__ __forceinline__ void race(Best &best, const float (&l)[N], const int (&index)[N],
                                         const bool (&keep)[N]) const {
        float e[N];
#pragma unroll
        for (int x = 0; x < N; ++x) e[x] = __ldg(noise + (keep[x] ? index[x] : 0));
#pragma unroll
        for (int x = 0; x < N; ++x) {
            if (!keep[x]) continue;
            const float w = weight_of(l[x], m, T);
            if (w >= min_p) best.offer(w / fmaxf(e[x], 1.17549435e-38f), index[x]);
        }
    }
};

// The cuts and the race among the peers' `have` tokens.  with_index(least, f) passes their logits and
// indices to f(logit, index), where it may leave out logits below `least`; race(least, keep) has
// those race for which keep(logit, index) holds.  mass: of which top-p takes its share, where that is not
// the mass of these tokens (0).  False where they do not hold top-p's cut, unless nothing below them
// is kept.
template <int kThreads, typename Peers, typename WithIndex, typename Race>
__device__ __forceinline__ bool choose(Shared<kThreads> &s, Peers peers, const Query &q, float range, u64 mass,
                                       u64 have, WithIndex with_index, Race race) {
    const Scale scale = {q.m, q.c};
    auto each = [&](uint32_t least, auto f) { with_index(key_logit(least), [&](float l, int) { f(l); }); };
    Cut cut = {0, 0xffffffffu};
    bool found = true;
    if (q.by_k && have > (u64)q.asked)
        cut = find_cut<kThreads>(s, peers, scale, range, false, q.by_p, q.asked, 0.0f, 0, &mass, &found, each);
    if (q.by_p) {
        const u64 target = max((u64)1, (u64)fmax(ceil((double)q.top_p * (double)mass), 0.0));
        u64 unused;
        const Cut at = find_cut<kThreads>(s, peers, scale, range, true, true, target,
                                          mass ? 0.0f : fmaxf(q.top_p, 1e-30f), cut.low, &unused, &found, each);
        // Less mass at hand: top-p's cut is below min_p's, or else below the list.
        if (found)
            cut = at.low == cut.low ? Cut{cut.low, min(cut.ties, at.ties)} : at;
        else if (!q.to_min)
            return false;
    }
    // Of the ties at the cut the lowest indices: the highest complements.
    uint32_t low_index = 0;
    if (cut.ties != 0xffffffffu) {
        u64 unused;
        low_index = cut_by_keys<kThreads>(s, peers, ~(uint32_t)(q.V - 1), 0xffffffffu, false, false, cut.ties, 0, 0,
                                          &unused, [&](auto f) {
            with_index(key_logit(cut.low), [&](float l, int i) {
                if (logit_key(l) == cut.low) f(~(uint32_t)i, []() { return (u64)0; });
            });
        }).low;
    }
    race(cut.low ? key_logit(cut.low) : kNegInf, [&](float l, int i) {
        const uint32_t k = logit_key(l);
        return l > kNegInf && (k > cut.low || (k == cut.low && ~(uint32_t)i >= low_index));
    });
    return true;
}

// f(vector, v) of a part's vectors in memory, four under way at a time.
template <int kThreads, typename T, typename F>
__device__ __forceinline__ void from_memory(const Part<T> &q, F f) {
    const int t = threadIdx.x, all = q.vecs();
#pragma unroll 1
    for (int v0 = t; v0 < all + t; v0 += 4 * kThreads) {
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = q.load(min(v0 + i * kThreads, all - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v0 + i * kThreads < all) f(u[i], v0 + i * kThreads);
    }
}
// f(vector, index of its first element) of the part, from shared memory where it is kept there.
template <int kThreads, bool kStaged, typename T, typename F>
__device__ __forceinline__ void each_vector(const Part<T> &part, const uint4 *copy, F f) {
    if (kStaged) {
        const int vecs = part.vecs();
#pragma unroll 2
        for (int v = threadIdx.x; v < vecs; v += kThreads) f(copy[v], part.index(v));
    } else {
        from_memory<kThreads>(part, [&](const uint4 &u, int v) { f(u, part.index(v)); });
    }
}

// Every block's best in its part, where the list does not do: `near`, the cuts are known to be among
// the tokens down to `edge`.  (Over 30 powers of two; scales that overflow take the histograms of
// keys.)
template <typename T, int kThreads, bool kStaged, typename Peers>
__device__ __forceinline__ u64 choose_from_all(Shared<kThreads> &s, Peers peers, const Query &q, const Part<T> &part,
                                               const uint4 *copy, bool near, float edge, u64 total, uint32_t n) {
    Best best;
    constexpr int kVec = Part<T>::kVec;
    auto on = [&](float l) { return !near || (l - q.m) * q.c >= -edge; };
    auto vectors = [&](float least, auto f) {
        each_vector<kThreads, kStaged>(part, copy, [&](const uint4 &u, int index) {
            const float top = max_of(u, T());
            if (top < least || (near && !on(top))) return;
            float e[kVec];
            unpack(u, e, T());
            f(e, index);
        });
    };
    choose<kThreads>(s, peers, q, near ? edge * 1.001f : 30.0f, near && !q.by_k ? total : 0, near ? n : q.V,
                     [&](float least, auto f) {
        vectors(least, [&](const float (&e)[kVec], int index) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (on(e[i])) f(fmaxf(e[i], kNegInf), index + i);
        });
    }, [&](float least, auto keep) {
        vectors(least, [&](const float (&e)[kVec], int index) {
            int at[kVec];
            bool in[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                at[i] = index + i;
                in[i] = e[i] >= least && on(e[i]) && keep(e[i], index + i);
            }
            q.race(best, e, at, in);
        });
    });
    return best.packed();
}

// kStaged: a block's part of a row fits shared memory.
template <typename T, int kThreads, bool kStaged>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(SampleParams p) {
    extern __shared__ __align__(16) unsigned char dynamic[];
    Shared<kThreads> &s = *reinterpret_cast<Shared<kThreads> *>(dynamic);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int row = blockIdx.x / C, t = threadIdx.x, V = p.vocab;
    // The blocks of a cluster may start at different times, and shared memory of one that has not
    // started may not be touched: the wait for this is before the first write to a peer's.
    if (C > 1) ptx::cluster_arrive_relaxed();
    const T *logits = static_cast<const T *>(p.logits) + row * p.logits_stride;
    const float *noise = p.noise + row * p.noise_stride;
    if (t == 0) {
        s.listed = s.locals = 0;
    }
    ptx::griddep_wait();
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    // (fmaxf: a NaN min-p keeps all, as 0 does.)
    const float min_p = p.min_p ? fmaxf(p.min_p[row], 0.0f) : 0.0f, top_p = p.top_p ? p.top_p[row] : 1.0f;
    const int asked = p.top_k ? p.top_k[row] : 0;
    const bool first_only = !(temp > 0.0f) || min_p > 1.0f || asked == 1;
    const bool by_k = asked > 0 && asked < V, by_p = top_p < 1.0f, by_min = min_p > 0.0f;
    const float T_ = temp > 0.0f ? temp : 1.0f, c = 1.44269504f / T_;

    // 1. This block's part, the maximum, and each thread's mass in weights of its own maximum so far
    // (while the memory is busy there is time for the exponentials).
    constexpr int kVec = Part<T>::kVec;
    auto part_of = [&](int from, int to) {
        Part<T> q;
        q.base = min(from, V);
        q.count = min(to, V) - q.base;
        const T *first = logits + q.base;
        q.skew = (int)(reinterpret_cast<uintptr_t>(first) % 16 / sizeof(T));
        q.at = first - q.skew;
        return q;
    };
    const Part<T> part = part_of(rank * p.chunk, (rank + 1) * p.chunk);
    static_assert(sizeof(Shared<kThreads>) % 16 == 0, "staged logits need 16-byte alignment");
    uint4 *const copy = reinterpret_cast<uint4 *>(dynamic + sizeof(Shared<kThreads>));
    float top_here = kNegInf, mass = 0.0f;
    const bool with_mass = by_p && !first_only;
    from_memory<kThreads>(part, [&](const uint4 &u, int v) {
        if (kStaged) copy[v] = u;
        const float top = fmaxf(max_of(u, T()), kNegInf);
        if (with_mass && top > kNegInf) {
            if (top > top_here) mass *= top_here > kNegInf ? pow2((top_here - top) * c) : 0.0f;
            top_here = fmaxf(top_here, top);
            float e[kVec];
            unpack(u, e, T());
#pragma unroll
            for (int i = 0; i < kVec; ++i) mass += pow2(fmaxf((e[i] - top_here) * c, -200.0f));
        }
        top_here = fmaxf(top_here, top);
    });
    uint32_t top_key = (uint32_t)block_max<kThreads>(logit_key(top_here), s.red);
    if (C > 1) {
        ptx::cluster_wait();
        if (t < C) cluster.map_shared_rank(&s, t)->tops[rank] = top_key;
        cluster.sync();
        for (int i = 0; i < C; ++i) top_key = max(top_key, s.tops[i]);
    } else {
        __syncthreads();
    }
    Shared<kThreads> *lead = C > 1 ? cluster.map_shared_rank(&s, 0) : &s;
    // The others have told the first block all that it needs: true where this block goes on alone.
    auto hand_over = [&]() {
        if (C == 1) {
            __syncthreads();
            return true;
        }
        ptx::cluster_arrive();
        if (rank != 0) return false;
        ptx::cluster_wait();
        return true;
    };
    const float m = key_logit(top_key);
    const bool greedy = first_only || m == kNegInf;
    Query q = {noise, m, c, T_, min_p, top_p, asked, V, by_k, by_p, false};
    Best best;
    if (greedy || !(by_k || by_p || by_min)) {
        each_vector<kThreads, kStaged>(part, copy, [&](const uint4 &u, int index) {
            if (greedy && !(max_of(u, T()) >= m)) return;
            float e[kVec];
            int at[kVec];
            bool in[kVec];
            unpack(u, e, T());
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                at[i] = index + i;
                in[i] = e[i] > kNegInf;
                if (greedy && e[i] == m) best.offer(0.0f, index + i);
            }
            if (!greedy) q.race(best, e, at, in);
        });
        u64 mine = block_max<kThreads>(best.packed(), s.red);
        if (t == 0) lead->bests[rank] = mine;
        if (!hand_over()) return;
        if (t == 0) {
            for (int i = 0; i < C; ++i) mine = max(mine, s.bests[i]);
            p.tokens[row] = m == kNegInf ? -1 : (int64_t)(uint32_t)~(uint32_t)mine;
        }
        return;
    }

    // 2. The mass and the list, in powers of two.  The list's edge lies a little below min_p's; with
    // top-k and top-p it is the far one, since top-p's share is of all the top-k tokens' mass.
    const float far = -log2f(min_p) * 1.00001f + 1e-4f;
    const bool to_min = by_min && far < kListBits && !(by_k && by_p);   // nothing below the list is kept
    const float edge = to_min ? far : kListBits;
    const bool usable = m < __builtin_inff() && c < __builtin_inff();
    if (usable) {
        each_vector<kThreads, kStaged>(part, copy, [&](const uint4 &u, int index) {
            if (!((max_of(u, T()) - m) * c >= -edge)) return;
            float e[kVec];
            unpack(u, e, T());
            int mine = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) mine += (e[i] - m) * c >= -edge;
            int at = atomicAdd(&s.locals, mine);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if ((e[i] - m) * c >= -edge) {
                    if (at < kLocalMax) s.local[at] = Listed{logit_key(e[i]), (uint32_t)(index + i)};
                    ++at;
                }
        });
        if (by_p) {
            const float share = top_here > kNegInf ? mass * pow2((top_here - m) * c) : 0.0f;
            const u64 total = block_sum<kThreads>(fixed_of(share), s.red);
            if (t == 0) lead->totals[rank] = total;
        }
        // This block's tokens to the first block's list; one that has too many spoils the list.
        __syncthreads();
        const uint32_t n = s.locals;
        if (t == 0) s.bin = atomicAdd(&lead->listed, n + (n > kLocalMax ? kSpoilt : 0)) % kSpoilt;
        __syncthreads();
        for (int i = t; i < min(n, (uint32_t)kLocalMax); i += kThreads)
            if (s.bin + i < kListMax) lead->list[s.bin + i] = s.local[i];
    }
    if (C > 1) cluster.sync(); else __syncthreads();

    u64 total = 0;
    const Shared<kThreads> &told = rank == 0 ? s : *lead;
    for (int i = 0; by_p && usable && i < C; ++i) total += told.totals[i];
    const uint32_t listed = told.listed, n = listed % kSpoilt;
    // 3. and 4.  The list holds the cuts if top-k's is inside; top-p's is looked for.
    q.to_min = to_min;
    const bool near = usable && (by_k ? n >= asked || (to_min && !by_p) : to_min);
    bool done = false;
    if (rank == 0 && usable && listed <= kListMax && (near || (by_p && !by_k)))
        done = choose<kThreads>(s, Alone(), q, edge * 1.001f, by_k ? 0 : total, n, [&](float, auto f) {
            for (int i = t; i < n; i += kThreads) f(key_logit(s.list[i].key), (int)s.list[i].index);
        }, [&](float, auto keep) {
            constexpr int kEach = 4;
            for (int i0 = t; i0 < n; i0 += kEach * kThreads) {
                float l[kEach];
                int at[kEach];
                bool in[kEach];
#pragma unroll
                for (int x = 0; x < kEach; ++x) {
                    const Listed &item = s.list[min(i0 + x * kThreads, (int)n - 1)];
                    l[x] = key_logit(item.key);
                    at[x] = (int)item.index;
                    in[x] = i0 + x * kThreads < n && keep(l[x], at[x]);
                }
                q.race(best, l, at, in);
            }
        });
    // The others have read the first block's totals when they arrive: it may not end before that, but
    // has its race to finish first where the list did.
    const bool to_wait = C > 1 && done;
    if (C > 1) {
        if (rank == 0 && t < C) cluster.map_shared_rank(&s, t)->wide = !done;
        ptx::cluster_arrive();
        if (!to_wait) {
            ptx::cluster_wait();
            if (!s.wide) return;
        }
    }
    u64 won = best.packed();
    if (!done)
        won = C > 1 ? choose_from_all<T, kThreads, kStaged>(s, Together{C}, q, part, copy, near, edge, total, n)
                    : choose_from_all<T, kThreads, kStaged>(s, Alone(), q, part, copy, near, edge, total, n);
    won = block_max<kThreads>(won, s.red);
    if (!done && C > 1) {
        if (t == 0) lead->bests[rank] = won;
        if (!hand_over()) return;
        for (int i = 0; i < C; ++i) won = max(won, s.bests[i]);
    }
    if (t == 0) p.tokens[row] = (int64_t)(uint32_t)~(uint32_t)won;
    if (to_wait) ptx::cluster_wait();
}

template <typename T, int kThreads, bool kStaged>
cudaError_t launch(const SampleParams &p, int rows, int cluster, cudaStream_t st) {
    const auto kernel = sample_kernel<T, kThreads, kStaged>;
    const size_t smem = sizeof(Shared<kThreads>) + (kStaged ? (size_t)p.chunk * sizeof(T) + 32 : 0);
    static PerDeviceOnce once;
    const cudaError_t e = once.run(current_device(), cudaSuccess, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(Shared<kThreads>) + kStageBytesAlone + 32);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t launch(const ctr_sampler_s *pl, SampleParams p, cudaStream_t st) {
    // Blocks a row: two an SM for few rows, but at least 4096 elements each.  A part that does not
    // fit shared memory is read again from L2: 256 rows of 100003 16-bit logits, one block a row, take
    // 33 us, and in clusters of four, whose parts fit but whose blocks wait for one another, 42.
    int cluster = 1;
    const int rows = (int)pl->rows;
    while (cluster < kMaxCluster && (int64_t)rows * cluster <= pl->num_sms && p.vocab >= 4096 * 2 * cluster)
        cluster *= 2;
    p.chunk = ((p.vocab + cluster - 1) / cluster + 15) / 16 * 16;
    if (p.chunk <= 4096) return launch<T, 256, true>(p, rows, cluster, st);
    // Where every block has an SM to itself more of a row fits: 1 row of 131072 fp32 logits, top-k 50, takes
    // 30 us so and 39 from L2.
    const bool alone = (int64_t)rows * cluster <= pl->num_sms;
    return (size_t)p.chunk * sizeof(T) <= (alone ? kStageBytesAlone : kStageBytes)
               ? launch<T, 512, true>(p, rows, cluster, st)
               : launch<T, 512, false>(p, rows, cluster, st);
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
    pl->num_sms = ctr::device_sms();
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
    ctr::SampleParams p = {};
    p.logits = logits;
    p.noise = noise;
    p.logits_stride = logits_stride;
    p.noise_stride = noise_stride;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.tokens = tokens;
    p.vocab = (int)pl->vocab;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = pl->dtype == CTR_F32    ? ctr::launch<float>(pl, p, st)
                          : pl->dtype == CTR_BF16 ? ctr::launch<__nv_bfloat16>(pl, p, st)
                                                  : ctr::launch<__half>(pl, p, st);
    return e == cudaSuccess ? CTR_OK : CTR_ERR_CUDA;
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
