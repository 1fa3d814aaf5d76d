// attention16.cuh -- attention of one new token over a paged cache of 16-bit rows.
//
// One query row reads every K and V row of its sequence once, 4 D bytes a slot and KV head for
// 4 D operations a query head: with G query heads to a KV head that is G operations a byte, so
// the cache's bytes bound it up to G of about 16 as long as the products run on the tensor
// pipe (on the CUDA cores the conversions and G multiply-adds an element would bound it from
// G = 4 on).  The heads of a group are the 16 rows of an m16n8k16 product, so a warp
// multiplies 16 query heads with 16 slots at a time; with fewer heads the spare rows cost tensor
// time only, of which a memory-bound kernel has plenty.  tcgen05 would want 128 rows: no
// group has them.
//
// Work: a unit is one sequence, KV head and set of 16 query heads; its slots come in tiles of
// 64, 16 to each of a block's four warps.  All tiles of all units in a row are cut into
// equal runs, one for each resident block, so ragged lengths and long sequences fill the GPU
// alike.  Every warp streams its own slots through a ring of cp.async stages without block
// barriers, and keeps a running maximum, sum and output of its own; the warps join once for
// each unit of the block's run.  A unit that several blocks share is joined by the
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
constexpr int kSlice = 16;              // output columns joined at a time
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

// Bytes between the rows of a stage: an odd number of 16-byte chunks, so that the eight rows of
// an ldmatrix lie in different banks (D is a multiple of 16).
__host__ __device__ inline int row_pitch(int D) { return 2 * D + 16; }
// Stages of a warp's ring.  Two blocks of 128 columns fit an SM with three stages of 8.5 KB to
// a warp: 139 KB in flight an SM, where 45 KB would cover 1 us of latency at full rate.
template <int DP> struct Ring { static constexpr int kStages = DP == 64 ? 5 : 3; };
template <int DP> inline size_t smem_bytes(int D, int B) {
    return (size_t)kWarps * Ring<DP>::kStages * 32 * row_pitch(D) +
           sizeof(float) * kWarps * 16 * (kSlice + 4) + 8 * (size_t)B + 64;
}

// A place in the row of all tiles: tile `tile` of head set hv of sequence b.
struct Place {
    int b, hv, tile, tiles, n, lo, first;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attention16_kernel(AttnParams p) {
    constexpr int S = Ring<DP>::kStages, KS = DP / 16, NT = DP / 8;
    typedef Pair<T> P;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red_m[kWarps][16], red_l[kWarps][16];
    __shared__ int64_t scan_total;
    __shared__ uint32_t slot_masks[kWarps][S];
    __shared__ int is_last;
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int pitch = row_pitch(p.D), stage_bytes = 32 * pitch;
    unsigned char *ring = smem + (size_t)warp * S * stage_bytes;
    float *merge = reinterpret_cast<float *>(smem + (size_t)kWarps * S * stage_bytes);
    int *prefix = reinterpret_cast<int *>(merge + kWarps * 16 * (kSlice + 4));   // [B]
    int *ntok = prefix + p.B;                                                      // [B]
    const bool with_new = p.k_new != nullptr;
    ptx::griddep_wait();

    // Tiles before each sequence (of one head set), and all of them.
    auto first_of = [&](int n) {
        return p.window > 0 && n > p.window ? (n - (int)p.window) / kTile * kTile : 0;
    };
    auto tiles_of = [&](int n) { return max(1, (n - first_of(n) + kTile - 1) / kTile); };
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
        int *warp_sum = reinterpret_cast<int *>(red_m);
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int base = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) base += warp_sum[i];
            all += warp_sum[i];
        }
        base += incl - sum;
        for (int b = b0; b < b1; ++b) {
            prefix[b] = base;
            base += tiles_of(abs(ntok[b]));
        }
        if (t == 0) scan_total = all;
        __syncthreads();
    }
    const int sets = (p.G + 15) / 16, Hu = p.Hkv * sets;
    const int64_t total = scan_total * Hu;
    const int64_t chunk = max((total + gridDim.x - 1) / gridDim.x, (int64_t)p.min_chunk);
    const int64_t t0 = chunk * blockIdx.x, t1 = min(t0 + chunk, total);
    if (t0 >= t1) return;

    auto enter = [&](Place &at) {
        at.n = abs(ntok[at.b]);
        at.lo = p.window > 0 && at.n > p.window ? at.n - (int)p.window : 0;
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

    // The producer side: where the next stage comes from, with its page number under way.
    Place in = use;
    int64_t to_issue = t1 - t0;
    int page_no = 0;
    auto page_index = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.cache.page; };
    auto fetch_page = [&]() {
        const int j = in.first + in.tile * kTile + warp * 16 + (lane & 15);
        page_no = j >= in.lo && j < in.n
                      ? __ldg(p.cache.tables + (int64_t)in.b * p.cache.table_pitch + page_index(j))
                      : -1;
    };
    const int chunks = p.D / 8;           // 16-byte chunks of a row
    auto issue = [&](int slot) {
        if (to_issue > 0) {
            const int j0 = in.first + in.tile * kTile + warp * 16, j = j0 + (lane & 15);
            const int hk = in.hv / sets;
            const bool inside = j >= in.lo && j < in.n;
            bool ok = inside && (unsigned)page_no < (unsigned)p.cache.num_pages;
            if (inside && !ok) atomicOr(p.cache.status, kStatusBadPage);
            int64_t off = 0;
            if (ok)
                off = page_no * p.cache.page_stride + hk * p.cache.head_stride +
                      (j - page_index(j) * p.cache.page) * p.cache.row_stride;
            const unsigned mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            if (lane == 0) slot_masks[warp][slot] = mask;
            const T *kp = static_cast<const T *>(p.k), *vp = static_cast<const T *>(p.v);
            // The row of the new token comes from the arguments, and goes to the cache.
            const bool newest = ntok[in.b] < 0 && j0 <= in.n - 1 && in.n - 1 < j0 + 16;
            const int new_row = newest ? in.n - 1 - j0 : -1;
            const int64_t new_off = in.b * p.kv_stride + (int64_t)hk * p.D;
            const uint32_t dst0 = ptx::smem_u32(ring + slot * stage_bytes);
            for (int i = 0; i < KS; ++i) {
                if (i * 16 >= p.D) break;
                const int c = i * 32 + lane, row = c / chunks, col = c - row * chunks;
                const int64_t o = __shfl_sync(0xffffffffu, off, row);
                const unsigned bytes = mask >> row & 1 ? 16 : 0;
                const T *ks = kp + o + col * 8, *vs = vp + o + col * 8;
                if (row == new_row && bytes) {
                    ks = static_cast<const T *>(p.k_new) + new_off + col * 8;
                    vs = static_cast<const T *>(p.v_new) + new_off + col * 8;
                    if (in.hv % sets == 0) {
                        *reinterpret_cast<uint4 *>(static_cast<T *>(p.k) + o + col * 8) =
                            *reinterpret_cast<const uint4 *>(ks);
                        *reinterpret_cast<uint4 *>(static_cast<T *>(p.v) + o + col * 8) =
                            *reinterpret_cast<const uint4 *>(vs);
                    }
                }
                const uint32_t dst = dst0 + row * pitch + col * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(ks),
                             "r"(bytes) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * pitch),
                             "l"(vs), "r"(bytes) : "memory");
            }
            --to_issue;
            if (to_issue > 0) {
                advance(in);
                fetch_page();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_page();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s);

    const int r0 = lane / 4, quad = lane % 4;
    int slot = 0;
    for (int64_t at = t0; at < t1;) {
        // One unit's share of this block's run.
        const int unit_b = use.b, hk = use.hv / sets, set = use.hv % sets;
        const int rows = min(16, p.G - set * 16);
        const int64_t h0 = (int64_t)hk * p.G + set * 16;     // its first query head
        const int64_t unit_start = (int64_t)prefix[use.b] * Hu + (int64_t)use.hv * use.tiles;
        const int64_t unit_end = unit_start + use.tiles, seg_end = min(unit_end, t1);
        const bool tall = rows > 8;
        uint32_t q[KS][4];
        {
            const T *qb = static_cast<const T *>(p.q) + unit_b * p.q_stride + h0 * p.D;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = r0 + (e & 1) * 8, d = i * 16 + (e >> 1) * 8 + quad * 2;
                    q[i][e] = row < rows && i * 16 < p.D
                                  ? __ldg(reinterpret_cast<const uint32_t *>(qb + row * p.D + d)) : 0u;
                }
        }
        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};

        for (const int64_t begin = at; at < seg_end; ++at) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();
            const uint32_t mask = slot_masks[warp][slot];
            issue(slot == 0 ? S - 1 : slot - 1);
            const uint32_t ks = ptx::smem_u32(ring + slot * stage_bytes), vs = ks + 16 * pitch;
            if (++slot == S) slot = 0;
            if (mask == 0 && !p.scores) continue;
            float s[2][4] = {};
            {
                const uint32_t a = ks + ((lane & 7) + (lane >> 4) * 8) * pitch + (lane >> 3 & 1) * 16;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (i * 16 >= p.D) break;
                    uint32_t b[4];
                    ldmatrix_x4(b, a + i * 32);
                    P::mma(s[0], q[i], b[0], b[1]);
                    P::mma(s[1], q[i], b[2], b[3]);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][e] *= p.scale_log2;
                    if (!(mask >> (x * 8 + quad * 2 + (e & 1)) & 1)) s[x][e] = kNegInf;
                }
            if (p.scores) {
                const int j = use.first + (int)(use.tile + (at - begin)) * kTile + warp * 16 + quad * 2;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = r0 + e * 8;
                    if (row >= rows) break;
                    float *dst = p.scores + ((int64_t)unit_b * p.Hq + h0 + row) * p.score_pitch + j;
                    // Whole pairs: the pitch is a multiple of 64 and covers every tile.
                    *reinterpret_cast<float2 *>(dst) = make_float2(s[0][e * 2], s[0][e * 2 + 1]);
                    *reinterpret_cast<float2 *>(dst + 8) = make_float2(s[1][e * 2], s[1][e * 2 + 1]);
                }
            }
            float shrink[2];
            bool grew = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = fmaxf(fmaxf(s[0][e * 2], s[0][e * 2 + 1]), fmaxf(s[1][e * 2], s[1][e * 2 + 1]));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                grew |= v > m[e];
                const float m2 = fmaxf(m[e], v);
                shrink[e] = m2 == kNegInf ? 1.0f : pow2(m[e] - m2);
                m[e] = m2;
            }
            if (__any_sync(0xffffffffu, grew)) {
                l[0] *= shrink[0];
                l[1] *= shrink[1];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][0] *= shrink[0];
                    o[i][1] *= shrink[0];
                    o[i][2] *= shrink[1];
                    o[i][3] *= shrink[1];
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (e == 1 && !tall) {
                    hi[1] = hi[3] = lo[1] = lo[3] = 0u;
                    break;
                }
                const float base = m[e] == kNegInf ? 0.0f : m[e];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float a = pow2(s[x][e * 2] - base), b = pow2(s[x][e * 2 + 1] - base);
                    l[e] += a + b;
                    const uint32_t h = P::pack(a, b);
                    const float2 f = P::unpack(h);
                    hi[x * 2 + e] = h;
                    lo[x * 2 + e] = P::pack(a - f.x, b - f.y);
                }
            }
            {
                const uint32_t a = vs + ((lane & 7) + (lane >> 3 & 1) * 8) * pitch + (lane >> 4) * 16;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (i * 16 >= p.D) break;
                    uint32_t b[4];
                    ldmatrix_x4_trans(b, a + i * 32);
                    P::mma(o[2 * i], hi, b[0], b[1]);
                    P::mma(o[2 * i + 1], hi, b[2], b[3]);
                    P::mma(o[2 * i], lo, b[0], b[1]);
                    P::mma(o[2 * i + 1], lo, b[2], b[3]);
                }
            }
        }

        // Join the four warps: the rows' maxima and sums, then the outputs slice by slice.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (quad == 0) {
                red_m[warp][r0 + e * 8] = m[e];
                red_l[warp][r0 + e * 8] = l[e];
            }
        }
        __syncthreads();
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = kNegInf;
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][r0 + e * 8]);
            f[e] = m[e] == kNegInf ? 0.0f : pow2(m[e] - top);
        }
        // This thread's row of the joined output, and its two columns of each slice.
        const int jr = t / 8, jc = t % 8 * 2;
        float top = kNegInf, sum = 0.0f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][jr]);
        for (int w = 0; w < kWarps; ++w)
            if (red_m[w][jr] != kNegInf) sum += red_l[w][jr] * pow2(red_m[w][jr] - top);
        const bool whole = at == unit_end && unit_start >= t0;
        const int64_t part = (int64_t)blockIdx.x * 2 + (max(unit_start, t0) == t0 ? 0 : 1);
        float *part_o = p.part_o + part * 16 * p.D;
        const int64_t head = (int64_t)unit_b * p.Hq + h0 + jr;
        for (int d0 = 0, i = 0; d0 < p.D; d0 += kSlice, ++i) {
#pragma unroll
            for (int k = 0; k < NT / 2; ++k)
                if (k == i) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float *dst = merge + (warp * 16 + r0) * (kSlice + 4) + x * 8 + quad * 2;
                        *reinterpret_cast<float2 *>(dst) =
                            make_float2(o[2 * k + x][0] * f[0], o[2 * k + x][1] * f[0]);
                        if (tall)
                            *reinterpret_cast<float2 *>(dst + 8 * (kSlice + 4)) =
                                make_float2(o[2 * k + x][2] * f[1], o[2 * k + x][3] * f[1]);
                    }
                }
            __syncthreads();
            if (jr < rows && d0 + jc < p.D) {
                float2 v = make_float2(0.f, 0.f);
                for (int w = 0; w < kWarps; ++w) {
                    const float2 u = *reinterpret_cast<const float2 *>(
                        merge + (w * 16 + jr) * (kSlice + 4) + jc);
                    v.x += u.x;
                    v.y += u.y;
                }
                if (whole) {
                    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
                    *reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + head * p.D + d0 + jc) =
                        P::pack(v.x * r, v.y * r);
                } else {
                    *reinterpret_cast<float2 *>(part_o + jr * p.D + d0 + jc) = v;
                }
            }
            __syncthreads();
        }
        if (jr < rows && jc == 0) {
            if (whole) {
                if (p.scores) p.stats[head] = make_float2(top, sum);
            } else {
                p.part_ml[part * 16 + jr] = make_float2(top, sum);
            }
        }
        if (!whole) {
            // The last block of the unit's to arrive joins the parts, in block order.
            const int64_t c0 = unit_start / chunk, c1 = (unit_end - 1) / chunk;
            __threadfence();
            __syncthreads();
            if (t == 0) {
                uint32_t *count = p.counters + (int64_t)unit_b * Hu + hk * sets + set;
                const uint32_t before = atomicAdd(count, 1u);
                is_last = before == (uint32_t)(c1 - c0);
                if (is_last) *count = 0;
            }
            __syncthreads();
            if (is_last) {
                __threadfence();
                const int64_t p0 = c0 * 2 + (unit_start == c0 * chunk ? 0 : 1);
                for (int x = t; x < rows * p.D / 4; x += kThreads) {
                    const int row = x / (p.D / 4), d = x % (p.D / 4) * 4;
                    float M = kNegInf, L = 0.0f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int64_t c = c0; c <= c1; c += 8) {
                        float2 ml[8];
                        float4 u[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const int64_t id = c + y > c1 ? -1 : c + y == c0 ? p0 : (c + y) * 2;
                            ml[y] = id < 0 ? make_float2(kNegInf, 0.0f) : __ldcg(p.part_ml + id * 16 + row);
                            u[y] = id < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : __ldcg(reinterpret_cast<const float4 *>(
                                                p.part_o + (id * 16 + row) * p.D + d));
                        }
                        float M2 = M;
#pragma unroll
                        for (int y = 0; y < 8; ++y) M2 = fmaxf(M2, ml[y].x);
                        const float shrink = M2 == kNegInf ? 1.0f : pow2(M - M2);
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
                    const int64_t hq = (int64_t)unit_b * p.Hq + h0 + row;
                    uint2 w = make_uint2(P::pack(v.x * r, v.y * r), P::pack(v.z * r, v.w * r));
                    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + hq * p.D + d) = w;
                    if (p.scores && d == 0) p.stats[hq] = make_float2(M, L);
                }
            }
        }
        // The next unit of the run.
        use.tile = use.tiles - 1;
        if (at < t1) advance(use);
    }
}

}  // namespace attn16
}  // namespace ctr
