// attention16.cuh -- attention of one new token over a paged cache of 16-bit rows.
//
// One query row reads every K and V row of its sequence once, 4 D bytes a slot and KV head for
// 4 D operations a query head: with G query heads to a KV head that is G operations a byte, so
// the cache's bytes bound it up to G of about 16 as long as the products run on the tensor
// pipe (on the CUDA cores the conversions and G multiply-adds an element would bound it from
// G = 4 on).  The transposed products keep the tensor work small: K [16 slots x 16] times the
// queries [16 x 8 heads], and V^T [16 columns x 16 slots] times the probabilities [16 slots x 8
// heads], in m16n8k16 steps, once for each eight heads of a group of up to sixteen.
// tcgen05 would want 128 rows of queries: no group has them.
//
// Work: a unit is one sequence, KV head and set of 8 or 16 query heads; its slots come in tiles of
// 64, 16 to each of a block's four warps.  All tiles of all units in a row are cut into
// equal runs, one for each resident block, so ragged lengths and long sequences fill the GPU
// alike.  Every warp streams its own slots through a ring of cp.async stages without block
// barriers, and keeps a running maximum, sum and output of its own; the warps join once for each
// unit of the block's run.  (Bulk copies, one a row as the pages want them, issue from one lane
// at a time: 655 instructions a step against 230, and 532 us for the full batch.)  A unit that several blocks share is joined by the
// last of them to finish, in block order, so the result does not depend on timing.
//
// Rounding: scores, statistics and outputs are fp32.  The probabilities enter the product with
// V as two 16-bit terms (the rounded value and what rounding left), so they keep at least 15
// bits; one term alone would add as much error as the rounding of the output does.
#pragma once

#include "decode_device.cuh"
#include "ptx.cuh"

namespace ctr {
namespace attn16 {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16 * kWarps;      // slots of one block step
constexpr float kNegInf = -__builtin_inff();

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// 2^x with a relative error of 2^-22; 0 at -inf.
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// The transpose of an 8x8 matrix of 16-bit values that lies two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// 16 bytes to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0) : "memory");
}

// Bytes between the rows of a stage: an odd number of 16-byte chunks, so that the eight rows of
// an ldmatrix lie in different banks (D is a multiple of 16).
__host__ __device__ inline int row_pitch(int D) { return 2 * D + 16; }
// Stages of a warp's ring.  Two blocks of 128 columns fit an SM with three stages of 8.5 KB to
// a warp: 139 KB in flight an SM, where 45 KB would cover 1 us of latency at full rate.
template <int DP> struct Ring { static constexpr int kStages = DP == 64 ? 5 : 3; };
// Output columns joined at a time, for NH sets of eight heads.
template <int NH> struct Join {
    static constexpr int kSlice = 64 / NH, kPitch = kSlice + 4;
    static constexpr int kBytes = (int)sizeof(float) * kWarps * 8 * NH * kPitch;
};
template <int DP, int NH> inline size_t smem_bytes(int D, int B) {
    return (size_t)kWarps * Ring<DP>::kStages * 32 * row_pitch(D) + Join<NH>::kBytes + 8 * (size_t)B;
}

// The parts of one unit, of blocks c0 .. c1, to its outputs.  A block's part of the unit that
// its run begins with is its first, else its second.
template <typename T>
__device__ __noinline__ void join_parts(const AttnParams &p, int64_t c0, int64_t c1, bool first_of_c0,
                                        int rows, int64_t h0) {
    const int quads = p.D / 4;
    for (int x = threadIdx.x; x < rows * quads; x += kThreads) {
        const int row = x / quads, d = x % quads * 4;
        float M = kNegInf, L = 0.0f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int64_t c = c0; c <= c1; c += 8) {
            float2 ml[8];
            float4 u[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int64_t id = c + y == c0 && !first_of_c0 ? c0 * 2 + 1 : (c + y) * 2;
                const bool on = c + y <= c1;
                ml[y] = on ? __ldcg(p.part_ml + id * 16 + row) : make_float2(kNegInf, 0.0f);
                u[y] = on ? __ldcg(reinterpret_cast<const float4 *>(p.part_o + (id * 16 + row) * p.D + d))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float M2 = M;
#pragma unroll
            for (int y = 0; y < 8; ++y) M2 = fmaxf(M2, ml[y].x);
            const float shrink = M == kNegInf ? 0.0f : pow2(M - M2);
            M = M2;
            L *= shrink;
            v.x *= shrink;
            v.y *= shrink;
            v.z *= shrink;
            v.w *= shrink;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float g = ml[y].x == kNegInf ? 0.0f : pow2(ml[y].x - M);
                L = fmaf(ml[y].y, g, L);
                v.x = fmaf(u[y].x, g, v.x);
                v.y = fmaf(u[y].y, g, v.y);
                v.z = fmaf(u[y].z, g, v.z);
                v.w = fmaf(u[y].w, g, v.w);
            }
        }
        const float r = L > 0.0f ? 1.0f / L : 0.0f;
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (h0 + row) * p.D + d) =
            make_uint2(Pair<T>::pack(v.x * r, v.y * r), Pair<T>::pack(v.z * r, v.w * r));
        if (p.scores && d == 0) p.stats[h0 + row] = make_float2(M, L);
    }
}

// A tile's place: tile `tile` of head set hv of sequence b.
struct Place {
    int b, hv, tile, tiles, n, lo, first;
};

// A running maximum is raised only when a score exceeds it by 2^kSlack: until then the
// probabilities may reach 2^kSlack, which changes no rounding, and the steps in between need no
// reduction over the warp.
constexpr float kSlack = 8.0f;

template <typename T, int DP, int NH>
__global__ void __launch_bounds__(kThreads) attention16_kernel(AttnParams p) {
    constexpr int S = Ring<DP>::kStages, KS = DP / 16, HN = 8 * NH;
    constexpr int kSlice = Join<NH>::kSlice, kPitch = Join<NH>::kPitch;
    typedef Pair<T> P;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t slot_masks[kWarps][S];
    __shared__ float red_m[kWarps][HN], red_l[kWarps][HN];
    __shared__ int warp_sum[kWarps];
    __shared__ int is_last;
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int pitch = row_pitch(p.D), stage_bytes = 32 * pitch;
    unsigned char *ring = smem + (size_t)warp * S * stage_bytes;
    float *merge = reinterpret_cast<float *>(smem + (size_t)kWarps * S * stage_bytes);
    int *prefix = reinterpret_cast<int *>(merge + kWarps * HN * kPitch);           // [B]
    int *ntok = prefix + p.B;                                                      // [B]
    const bool with_new = p.k_new != nullptr;
    ptx::griddep_wait();

    // Tiles before each sequence (of one head set), and all of them.
    auto lo_of = [&](int n) { return p.window > 0 && n > p.window ? n - (int)p.window : 0; };
    auto tiles_of = [&](int n) { return max(1, (n + kTile - 1) / kTile - lo_of(n) / kTile); };
    int64_t total;
    const int sets = (p.G + HN - 1) / HN, Hu = p.Hkv * sets;
    {
        const int per = (p.B + kThreads - 1) / kThreads, b0 = min(t * per, p.B),
                  b1 = min(b0 + per, p.B);
        int sum = 0, len;
        for (int b = b0; b < b1; ++b) {
            const int n = tokens_of(p.cache, b, with_new, &len);
            // The sign says whether the last token is the new one.
            ntok[b] = with_new && n > len && len >= 0 ? -n : n;
            sum += tiles_of(n);
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int base = incl - sum, all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) base += warp_sum[i];
            all += warp_sum[i];
        }
        for (int b = b0; b < b1; ++b) {
            prefix[b] = base;
            base += tiles_of(abs(ntok[b]));
        }
        total = (int64_t)all * Hu;
        __syncthreads();
    }
    const int64_t chunk = max((total + gridDim.x - 1) / gridDim.x, (int64_t)p.min_chunk);
    const int64_t t0 = chunk * blockIdx.x, t1 = min(t0 + chunk, total);
    if (t0 >= t1) return;

    auto enter = [&](Place &at) {
        at.n = abs(ntok[at.b]);
        at.lo = lo_of(at.n);
        at.first = at.lo / kTile * kTile;
        at.tiles = tiles_of(at.n);
    };
    auto advance = [&](Place &at) {
        if (++at.tile == at.tiles) {
            at.tile = 0;
            if (++at.hv == Hu) {
                at.hv = 0;
                if (++at.b < p.B) enter(at);
            }
        }
    };
    Place use;
    {
        const int x = (int)(t0 / Hu);
        int lo = 0, hi = p.B - 1;        // the last sequence with prefix <= x
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
        }
        use.b = lo;
        enter(use);
        const int64_t rem = t0 - (int64_t)prefix[lo] * Hu;
        use.hv = (int)(rem / use.tiles);
        use.tile = (int)(rem % use.tiles);
    }

    // The producer side: kLanes lanes copy a row, 16 bytes each, kRows rows at a time.
    constexpr int kLanes = DP / 8, kRows = 32 / kLanes;
    Place in = use;
    int64_t to_issue = t1 - t0;
    const int row0 = lane / kLanes, col = lane % kLanes;
    const bool copies = col * 8 < p.D;
    // With pages of whole sixteens a warp's slots lie in one page.
    const bool one_page = p.cache.page % 16 == 0;
    const int64_t lane_off = (one_page ? row0 * p.cache.row_stride : 0) + col * 8;
    const int64_t row_step = kRows * p.cache.row_stride;
    const uint32_t lane_dst = ptx::smem_u32(ring) + row0 * pitch + col * 16;
    int page_no = 0;           // of slot (lane & 15) of the next stage, under way
    auto page_index = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.cache.page; };
    auto fetch_page = [&]() {
        const int j = in.first + in.tile * kTile + warp * 16 + (lane & 15);
        page_no = j >= in.lo && j < in.n
                      ? __ldg(p.cache.tables + (int64_t)in.b * p.cache.table_pitch + page_index(j))
                      : -1;
    };
    auto issue = [&](int slot) {
        if (to_issue > 0) {
            const int j0 = in.first + in.tile * kTile + warp * 16, j = j0 + (lane & 15);
            const int hk = sets == 1 ? in.hv : in.hv / sets;
            const bool ok = (unsigned)page_no < (unsigned)p.cache.num_pages;
            const unsigned mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            int64_t off = page_no * p.cache.page_stride + hk * p.cache.head_stride +
                          (j - page_index(j) * p.cache.page) * p.cache.row_stride;
            if (lane == 0) slot_masks[warp][slot] = mask;
            if (mask != 0xffffu && !ok && j >= in.lo && j < in.n)
                atomicOr(p.cache.status, kStatusBadPage);
            const uint32_t dst = lane_dst + slot * stage_bytes;
            const int newest = ntok[in.b];       // -n where slot n - 1 is the new token's
            if (mask == 0xffffu && one_page && !(newest < 0 && -newest - 1 < j0 + 16)) {
                off = __shfl_sync(0xffffffffu, off, 0) + lane_off;
                const T *ks = static_cast<const T *>(p.k) + off, *vs = static_cast<const T *>(p.v) + off;
                if (copies) {
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        copy16(dst + i * kRows * pitch, ks, true);
                        copy16(dst + (16 + i * kRows) * pitch, vs, true);
                        ks += row_step;
                        vs += row_step;
                    }
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < KS; ++i) {
                    const int row = i * kRows + row0;
                    const int64_t o = __shfl_sync(0xffffffffu, off, row) + col * 8;
                    const bool on = mask >> row & 1;
                    const T *ks = static_cast<const T *>(p.k) + o, *vs = static_cast<const T *>(p.v) + o;
                    if (!copies) continue;
                    if (on && newest == -(j0 + row + 1)) {
                        // The new token's row comes from the arguments, and goes to the cache.
                        const int64_t x = in.b * p.kv_stride + (int64_t)hk * p.D + col * 8;
                        T *kc = const_cast<T *>(ks), *vc = const_cast<T *>(vs);
                        ks = static_cast<const T *>(p.k_new) + x;
                        vs = static_cast<const T *>(p.v_new) + x;
                        if (in.hv == hk * sets) {
                            *reinterpret_cast<uint4 *>(kc) = *reinterpret_cast<const uint4 *>(ks);
                            *reinterpret_cast<uint4 *>(vc) = *reinterpret_cast<const uint4 *>(vs);
                        }
                    }
                    // Hidden slots are filled with zeros: no probability is given to them, and
                    // what V holds there must be finite.  (The address is not read.)
                    copy16(dst + i * kRows * pitch, on ? ks : p.k, on);
                    copy16(dst + (16 + i * kRows) * pitch, on ? vs : p.v, on);
                }
            }
            if (--to_issue > 0) {
                advance(in);
                fetch_page();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_page();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) issue(s);

    const int r0 = lane / 4, quad = lane % 4;
    int slot = 0;
    for (int64_t at = t0; at < t1;) {
        // One unit's share of this block's run.
        const int hk = use.hv / sets, set = use.hv % sets;
        const int rows = min(HN, p.G - set * HN);
        const int64_t h0 = (int64_t)use.b * p.Hq + (int64_t)hk * p.G + set * HN;   // first query head
        const int64_t unit_start = (int64_t)prefix[use.b] * Hu + (int64_t)use.hv * use.tiles;
        const int64_t unit_end = unit_start + use.tiles;
        const int steps = (int)(min(unit_end, t1) - at);
        // Queries as the products' second operand: heads r0 (and r0 + 8), columns quad * 2.
        uint32_t q[NH][KS][2];
        {
            const T *qb = static_cast<const T *>(p.q) + use.b * p.q_stride +
                          ((int64_t)hk * p.G + set * HN) * p.D;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        q[h][i][e] = h * 8 + r0 < rows && i * 16 < p.D
                                         ? __ldg(reinterpret_cast<const uint32_t *>(
                                               qb + (h * 8 + r0) * p.D + i * 16 + e * 8 + quad * 2))
                                         : 0u;
        }
        float o[NH][KS][4];      // columns i * 16 + r0 (+ 8) of heads quad * 2 (+ 1)
        float m[NH][2], l[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h][0] = m[h][1] = kNegInf;
            l[h][0] = l[h][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[h][i][0] = o[h][i][1] = o[h][i][2] = o[h][i][3] = 0.0f;
        }
        for (int step = 0; step < steps; ++step) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();
            const uint32_t mask = slot_masks[warp][slot];
            issue(slot == 0 ? S - 1 : slot - 1);
            const uint32_t ks = ptx::smem_u32(ring + slot * stage_bytes), vs = ks + 16 * pitch;
            if (++slot == S) slot = 0;
            if (mask == 0 && !p.scores) continue;
            float s[NH][4] = {};     // slots r0 (+ 8 from the third) of heads quad * 2 (+ 1)
            {
                const uint32_t a = ks + ((lane & 7) + (lane >> 3 & 1) * 8) * pitch + (lane >> 4) * 16;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (i * 16 >= p.D) break;
                    uint32_t k[4];
                    ldmatrix_x4(k, a + i * 32);
#pragma unroll
                    for (int h = 0; h < NH; ++h) P::mma(s[h], k, q[h][i][0], q[h][i][1]);
                }
            }
            bool grew = false;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[h][e] *= p.scale_log2;
            if (mask != 0xffffu) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(mask >> (r0 + (e >> 1) * 8) & 1)) {
#pragma unroll
                        for (int h = 0; h < NH; ++h) s[h][e] = kNegInf;
                    }
            }
            if (p.scores) {
                // The pitch covers whole tiles.
                float *dst = p.scores + h0 * p.score_pitch + use.first + (use.tile + step) * kTile +
                             warp * 16 + r0;
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int head = h * 8 + quad * 2 + (e & 1);
                        if (head < rows) dst[head * p.score_pitch + (e >> 1) * 8] = s[h][e];
                    }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    grew |= fmaxf(s[h][e], s[h][e + 2]) > m[h][e] + kSlack;
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(s[h][e], s[h][e + 2]);
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        v = fmaxf(v, m[h][e]);
                        const float shrink = m[h][e] == kNegInf ? 0.0f : pow2(m[h][e] - v);
                        m[h][e] = v;
                        l[h][e] *= shrink;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[h][i][e] *= shrink;
                            o[h][i][e + 2] *= shrink;
                        }
                    }
            }
            uint32_t hi[NH][2], lo[NH][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                // A head without any slot so far has no maximum yet: its weights are 0.
                const float b0 = m[h][0] == kNegInf ? 0.0f : m[h][0];
                const float b1 = m[h][1] == kNegInf ? 0.0f : m[h][1];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = pow2(s[h][2 * e] - b0), y = pow2(s[h][2 * e + 1] - b1);
                    l[h][0] += x;
                    l[h][1] += y;
                    const uint32_t r = P::pack(x, y);
                    const float2 f = P::unpack(r);
                    hi[h][e] = transpose8(r);
                    lo[h][e] = transpose8(P::pack(x - f.x, y - f.y));
                }
            }
            {
                const uint32_t a = vs + ((lane & 7) + (lane >> 4) * 8) * pitch + (lane >> 3 & 1) * 16;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (i * 16 >= p.D) break;
                    uint32_t v[4];
                    ldmatrix_x4_trans(v, a + i * 32);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        P::mma(o[h][i], v, hi[h][0], hi[h][1]);
                        P::mma(o[h][i], v, lo[h][0], lo[h][1]);
                    }
                }
            }
        }
        at += steps;

        // Join the four warps: the heads' maxima and sums, then the outputs slice by slice.
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[h][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (r0 == 0) {
                    red_m[warp][h * 8 + quad * 2 + e] = m[h][e];
                    red_l[warp][h * 8 + quad * 2 + e] = v;
                }
            }
        __syncthreads();
        float f[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = kNegInf;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][h * 8 + quad * 2 + e]);
                f[h][e] = m[h][e] == kNegInf ? 0.0f : pow2(m[h][e] - top);
            }
        // This thread's head of the joined output, and its four columns of each slice.
        const int jh = t / (kSlice / 4), jc = t % (kSlice / 4) * 4;
        float top = kNegInf, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][jh]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (red_m[w][jh] != kNegInf) sum += red_l[w][jh] * pow2(red_m[w][jh] - top);
        const bool whole = at == unit_end && unit_start >= t0;
        const int64_t part = (int64_t)blockIdx.x * 2 + (unit_start <= t0 ? 0 : 1);
        float *part_o = p.part_o + part * 16 * p.D;
#pragma unroll
        for (int k = 0; k < DP / kSlice; ++k) {
            const int d0 = k * kSlice;
            if (d0 >= p.D) break;
#pragma unroll
            for (int x = 0; x < kSlice / 16; ++x)
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        merge[(warp * HN + h * 8 + quad * 2 + (e & 1)) * kPitch + x * 16 + r0 +
                              (e >> 1) * 8] = o[h][k * (kSlice / 16) + x][e] * f[h][e & 1];
            __syncthreads();
            if (jh < rows && d0 + jc < p.D) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 u = *reinterpret_cast<const float4 *>(merge + (w * HN + jh) * kPitch + jc);
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
                if (whole) {
                    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
                    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (h0 + jh) * p.D + d0 + jc) =
                        make_uint2(P::pack(v.x * r, v.y * r), P::pack(v.z * r, v.w * r));
                } else {
                    *reinterpret_cast<float4 *>(part_o + jh * p.D + d0 + jc) = v;
                }
            }
            __syncthreads();
        }
        if (jh < rows && jc == 0) {
            if (!whole)
                p.part_ml[part * 16 + jh] = make_float2(top, sum);
            else if (p.scores)
                p.stats[h0 + jh] = make_float2(top, sum);
        }
        if (!whole) {
            // The last block of the unit's to arrive joins the parts, in block order.
            const int64_t c0 = unit_start / chunk, c1 = (unit_end - 1) / chunk;
            __threadfence();
            __syncthreads();
            if (t == 0) {
                uint32_t *count = p.counters + (int64_t)use.b * Hu + use.hv;
                is_last = atomicAdd(count, 1u) == (uint32_t)(c1 - c0);
                if (is_last) *count = 0;
            }
            __syncthreads();
            if (is_last) {
                __threadfence();
                join_parts<T>(p, c0, c1, unit_start == c0 * chunk, rows, h0);
            }
        }
        // The next unit of the run.
        use.tile = use.tiles - 1;
        if (at < t1) advance(use);
    }
}

}  // namespace attn16
}  // namespace ctr
