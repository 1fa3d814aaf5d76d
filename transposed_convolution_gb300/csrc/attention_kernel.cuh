// attention_kernel.cuh -- attention of one new token over a paged cache.
//
// One query row reads every K and V row of its sequence once, 4 D bytes (16-bit caches) a slot and KV
// head for 4 D operations a query head: with G query heads to a KV head that is G operations a
// byte, so the cache's bytes bound it up to G of about 16 as long as the products run on the
// tensor pipe (on the CUDA cores the conversions and G multiply-adds an element would bound it
// from G = 4 on).  The transposed products keep the tensor work small: K [16 slots x 16] times
// the queries [16 x 8 heads], and V^T [16 columns x 16 slots] times the probabilities [16 slots x
// 8 heads], in m16n8k16 steps, once for each eight heads of a group of up to sixteen.
// tcgen05 would want 128 rows of queries: no group has them.  fp32 caches have twice the
// bytes for the same operations, and their sums stay fp32 multiply-adds on the CUDA cores: the tensor
// pipe's own accumulation, even of tf32 terms that add up to fp32, drifts over a long row.
//
// Work: a unit is one sequence, KV head and set of 8 or 16 query heads; its slots come in tiles,
// 16 to each of a block's warps.  All units' tiles, in a row, are cut into equal chunks, one for
// each resident block, so ragged lengths and long sequences fill the GPU alike; entering a
// unit counts as one tile more.  The parts of a unit that several chunks share are joined in
// chunk order by a second kernel, whose launch overlaps the first one's end, so the result does
// not depend on timing.  (Joined by the last block to arrive, behind a fence and a counter, two
// parts took 3.4 us and 33 parts 7.)  Caches of up to kWholeSlots slots are cut into whole
// units, without a second kernel.  Each set of a larger group is a unit of its own and reads its K and V
// again: 16 sequences of 8192 slots, 2 KV heads of 128, take 30 us for 8 query heads to a KV head in bf16,
// 36 for 16, 54 for 32 and 91 for 64; in fp32, with sets of 8, 59, 105, 193 and 369.  A queue of small chunks for the last quarter, for blocks that
// run ahead, gained less than its parts cost once the rings were as short as they are.
//
// Every warp streams its own slots through a ring of cp.async stages without block barriers,
// and keeps a running base, sum and output of its own; the warps join once for each unit of
// a chunk.  (Bulk copies, one a row as the pages want them, issue from one lane at a time:
// 655 instructions a step, and 532 us for the full batch.)
//
// Rounding: scores, statistics and outputs are fp32.  The probabilities enter the product with
// V as two 16-bit terms (the value rounded towards zero and what that left), so they keep at least 15
// bits; one term alone would add as much error as the rounding of the output does.  Neither term is
// negative or, unless the probability is, 0: an infinite value in V stays that infinity.
// fp16 terms end at 2^-24, which the lift (below) makes 2^-37 of the largest weight: probabilities of less
// than 2^-22 of that have fewer bits.  (Without the lift 2^-24 was all there was, and slots 17 nats under a
// warp's largest were left out.  The ragged fp16 batch takes 32.0 us with it and 31.8 without.)
#pragma once

#include "decode_device.cuh"
#include "ptx.cuh"

namespace ctr {
namespace attn {

constexpr float kNegInf = -__builtin_inff();

// Launch shapes by element size and largest head size: warps a block, stages of a warp's ring, and
// most blocks an SM.  What matters is warps an SM (each is held up by its own chain of products and
// exponentials) and short rings: with 70 KB in flight an SM, 128 columns of 16 bits, 131072 slots
// took 92 us; with 140 KB 102 us, because the blocks then ran less evenly; 45 KB would cover
// 1 us of latency.
template <int kBytes, int DP> struct Shape;
template <> struct Shape<2, 64> { static constexpr int kWarps = 4, kStages = 3, kPerSm = 4; };
template <> struct Shape<2, 128> { static constexpr int kWarps = 4, kStages = 2, kPerSm = 3; };
template <> struct Shape<2, 256> { static constexpr int kWarps = 6, kStages = 2, kPerSm = 1; };
template <> struct Shape<4, 64> { static constexpr int kWarps = 4, kStages = 2, kPerSm = 3; };
template <> struct Shape<4, 96> { static constexpr int kWarps = 4, kStages = 2, kPerSm = 2; };
template <> struct Shape<4, 128> { static constexpr int kWarps = 3, kStages = 2, kPerSm = 2; };
template <> struct Shape<4, 256> { static constexpr int kWarps = 3, kStages = 2, kPerSm = 1; };

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static constexpr float kLift = 0.0f, kSlack = 8.0f;
    static constexpr float kLeast = 1.17549435e-38f;      // smallest term (2^-126)
    // Rounded towards zero.
    static __device__ __forceinline__ uint32_t pack_down(float a, float b) {
        uint32_t r;
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
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
    static constexpr float kLift = 13.0f, kSlack = 2.0f;
    static constexpr float kLeast = 5.96046448e-8f;       // smallest term (2^-24)
    static __device__ __forceinline__ uint32_t pack_down(float a, float b) {
        uint32_t r;
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
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

// Four values to the output, rounded to its type.
template <typename T> __device__ __forceinline__ void store4(T *to, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(Pair<T>::pack(a, b), Pair<T>::pack(c, d));
}
__device__ __forceinline__ void store4(float *to, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(to) = make_float4(a, b, c, d);
}

// The first slot that n tokens attend to, and the tiles they take (one at least).
__device__ __forceinline__ int first_slot(const AttnParams &p, int n) {
    return p.window > 0 && n > p.window ? n - (int)p.window : 0;
}
template <int kTile> __device__ __forceinline__ int unit_tiles(const AttnParams &p, int n) {
    return max(1, (n + kTile - 1) / kTile - first_slot(p, n) / kTile);
}

// A walk over the units of a block's chunk (or, with whole units, over the block's units).
struct Walk {
    int x, x1;               // place in the chunk and its end
    int b, hv;               // unit
    int n, lo, first, tiles; // its sequence's
    int unit;                // the unit's place: its entry, then its tiles
    int tile, left;          // segment: next tile, and tiles left
    int count;               // segments (whole units) so far
};

// Weights are powers of two of a score's distance to its head's base, which follows the running maximum:
// it is raised, to kLift below the maximum, only when a score exceeds that maximum by kSlack.  Until
// then weights may reach 2^(kLift + kSlack), and the steps in between need no reduction over the warp.
// fp32 and bf16 weights have exponents to spare on either side.  fp16 ones end at 2^-24, so they are
// lifted to just below that type's largest: 2^15 for a slack of two, with the base rounded upwards, so that
// they stay below it for scores so large that the lift itself is rounded.
constexpr float kSlack = 8.0f;

// The arithmetic of one warp on 16 slots and up to kHeads heads, 16-bit types: lane (r0 = lane / 4,
// quad = lane % 4) has the scores of slots r0 and r0 + 8 for heads quad * 2 and quad * 2 + 1 of each
// eight, and the outputs of columns r0 and r0 + 8 of each sixteen.  kD is the head size, or 0 for
// any up to DP.
template <typename T, int DP, int NH, int kD_> struct Heads16 {
    typedef T Element;
    typedef Pair<T> P;
    typedef attn::Shape<2, DP> Shape;
    static constexpr int kMax = DP, kD = kD_, kHeads = 8 * NH, KS = DP / 16;
    static constexpr bool kSharedQueries = false;
    static constexpr int kSharedBytes = 0;
    // Bytes between the rows of a stage: an odd number of 16-byte chunks, so that the eight rows of
    // an ldmatrix lie in different banks (D is a multiple of 16).
    static __host__ __device__ int k_pitch(int D) { return 2 * D + 16; }
    static __host__ __device__ int v_pitch(int D) { return 2 * D + 16; }

    uint32_t q[NH][KS][2];   // the products' second operand: heads r0 (and r0 + 8), columns quad * 2
    float o[NH][KS][4], m[NH][2], l[NH][2];

    __device__ __forceinline__ void load_queries(const T *from, int rows, int D, unsigned char *) {
        const int lane = threadIdx.x % 32, r0 = lane / 4, quad = lane % 4;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    q[h][i][e] = h * 8 + r0 < rows && i * 16 < D
                                     ? *reinterpret_cast<const uint32_t *>(
                                           from + (h * 8 + r0) * D + i * 16 + e * 8 + quad * 2)
                                     : 0u;
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h][0] = m[h][1] = kNegInf;
            l[h][0] = l[h][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[h][i][0] = o[h][i][1] = o[h][i][2] = o[h][i][3] = 0.0f;
        }
    }

    // One stage: K and V rows of 16 slots, those of `mask` to be attended to.  scores: where head 0's
    // score of the first slot goes, or null.
    __device__ __forceinline__ void step(const unsigned char *k_rows, const unsigned char *v_rows,
                                         unsigned mask, int D, float scale_log2, int rows, float *scores,
                                         int64_t score_pitch, unsigned char *) {
        const int lane = threadIdx.x % 32, r0 = lane / 4, quad = lane % 4;
        const int pitch = k_pitch(D);
        float s[NH][4] = {};     // slots r0 (+ 8 from the third) of heads quad * 2 (+ 1)
        {
            const uint32_t a = ptx::smem_u32(k_rows) + ((lane & 7) + (lane >> 3 & 1) * 8) * pitch +
                               (lane >> 4) * 16;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                if (i * 16 >= D) break;
                uint32_t k[4];
                ldmatrix_x4(k, a + i * 32);
#pragma unroll
                for (int h = 0; h < NH; ++h) P::mma(s[h], k, q[h][i][0], q[h][i][1]);
            }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][e] *= scale_log2;
        if (mask != 0xffffu) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(mask >> (r0 + (e >> 1) * 8) & 1)) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) s[h][e] = kNegInf;
                }
        }
        if (scores) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int head = h * 8 + quad * 2 + (e & 1);
                    if (head < rows) scores[head * score_pitch + r0 + (e >> 1) * 8] = s[h][e];
                }
        }
        bool grew = false;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) grew |= fmaxf(s[h][e], s[h][e + 2]) > __fadd_rd(m[h][e], P::kLift + P::kSlack);
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[h][e], s[h][e + 2]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    v = fmaxf(__fsub_ru(v, P::kLift), m[h][e]);
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
            // A head without any slot so far has no base yet: its weights are 0.
            const float b0 = m[h][0] == kNegInf ? 0.0f : m[h][0];
            const float b1 = m[h][1] == kNegInf ? 0.0f : m[h][1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = pow2(s[h][2 * e] - b0), y = pow2(s[h][2 * e + 1] - b1);
                l[h][0] += x;
                l[h][1] += y;
                const uint32_t r = P::pack_down(x, y);
                const float2 f = P::unpack(r);
                hi[h][e] = transpose8(r);
                lo[h][e] = transpose8(P::pack(fmaxf(x - f.x, P::kLeast), fmaxf(y - f.y, P::kLeast)));
            }
        }
        const uint32_t a = ptx::smem_u32(v_rows) + ((lane & 7) + (lane >> 4) * 8) * pitch +
                           (lane >> 3 & 1) * 16;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            if (i * 16 >= D) break;
            uint32_t v[4];
            ldmatrix_x4_trans(v, a + i * 32);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                P::mma(o[h][i], v, hi[h][0], hi[h][1]);
                P::mma(o[h][i], v, lo[h][0], lo[h][1]);
            }
        }
    }

    // The warp's bases, sums and outputs [kHeads][pitch] to shared memory.
    __device__ __forceinline__ void put(float *red_m, float *red_l, float *to, int pitch, int D) {
        const int lane = threadIdx.x % 32, r0 = lane / 4, quad = lane % 4;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[h][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int head = h * 8 + quad * 2 + e;
                if (r0 == 0) {
                    red_m[head] = m[h][e];
                    red_l[head] = v;
                }
                float *row = to + head * pitch + r0;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (i * 16 >= D) break;
                    row[i * 16] = o[h][i][e];
                    row[i * 16 + 8] = o[h][i][e + 2];
                }
            }
    }
};

// The same for fp32 and H = 2 or 8 heads, on the CUDA cores.  Scores: lane (sg = lane / 4, dq = lane %
// 4) multiplies slots sg and sg + 8 with all heads over every fourth 16 bytes of the columns; the
// four lanes of a slot then exchange halves of what they have until each has the sums of its H / 2 of the
// 2 H (head, slot) pairs, pair x being head x / 2 and slot sg + 8 (x % 2).  Outputs: lane i has
// columns 4 i (and 4 i + 128) of all heads, and reads the probabilities from shared memory, as the
// queries: both are the same for many lanes, so they take no bandwidth to speak of.
template <int DP, int H, int kD_> struct Heads32 {
    typedef float Element;
    typedef attn::Shape<4, DP> Shape;
    static constexpr int kMax = DP, kD = kD_, kHeads = H, kOwn = H / 2, kCols = DP > 128 ? 2 : 1;
    static constexpr bool kSharedQueries = true;
    // The queries [H][DP], and each warp's probabilities [16][H].
    static constexpr int kSharedBytes = 4 * (H * DP + Shape::kWarps * 16 * H);
    // The rows of two neighbouring slots lie 16 banks apart in K.
    static __host__ __device__ int k_pitch(int D) { return 4 * (D + (D % 32 ? 0 : 16)); }
    static __host__ __device__ int v_pitch(int D) { return 4 * D; }

    float o[H][kCols][4], m[kOwn > 1 ? kOwn / 2 : 1], l[kOwn > 1 ? kOwn / 2 : 1];
    static constexpr int kMine = kOwn > 1 ? kOwn / 2 : 1;      // heads a lane owns pairs of

    __device__ __forceinline__ void load_queries(const float *from, int rows, int D, unsigned char *shared) {
        float *q = reinterpret_cast<float *>(shared);
        for (int x = threadIdx.x; x < H * DP; x += blockDim.x) {
            const int h = x / DP, d = x % DP;
            q[x] = h < rows && d < D ? from[h * D + d] : 0.0f;
        }
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            m[i] = kNegInf;
            l[i] = 0.0f;
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[h][c][0] = o[h][c][1] = o[h][c][2] = o[h][c][3] = 0.0f;
    }

    __device__ __forceinline__ void step(const unsigned char *k_rows, const unsigned char *v_rows,
                                         unsigned mask, int D, float scale_log2, int rows, float *scores,
                                         int64_t score_pitch, unsigned char *shared) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sg = lane / 4, dq = lane % 4;
        const float *q = reinterpret_cast<const float *>(shared) + dq * 4;
        float *prob = reinterpret_cast<float *>(shared) + H * DP + warp * 16 * H;
        float s[2 * H];
#pragma unroll
        for (int x = 0; x < 2 * H; ++x) s[x] = 0.0f;
        {
            const unsigned char *a = k_rows + sg * k_pitch(D) + dq * 16;
            const unsigned char *b = a + 8 * k_pitch(D);
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                if (j * 16 >= D) break;
                const float4 u = *reinterpret_cast<const float4 *>(a + j * 64);
                const float4 v = *reinterpret_cast<const float4 *>(b + j * 64);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float4 w = *reinterpret_cast<const float4 *>(q + h * DP + j * 16);
                    s[2 * h] = fmaf(u.w, w.w, fmaf(u.z, w.z, fmaf(u.y, w.y, fmaf(u.x, w.x, s[2 * h]))));
                    s[2 * h + 1] = fmaf(v.w, w.w, fmaf(v.z, w.z, fmaf(v.y, w.y, fmaf(v.x, w.x, s[2 * h + 1]))));
                }
            }
        }
        // Halves to the lane two off, then to the next: pairs [dq * kOwn, (dq + 1) * kOwn) remain.
        float half[H], mine[kOwn];
#pragma unroll
        for (int x = 0; x < H; ++x) {
            const float send = dq & 2 ? s[x] : s[H + x], keep = dq & 2 ? s[H + x] : s[x];
            half[x] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
        }
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
            const float send = dq & 1 ? half[x] : half[kOwn + x], keep = dq & 1 ? half[kOwn + x] : half[x];
            mine[x] = (keep + __shfl_xor_sync(0xffffffffu, send, 1)) * scale_log2;
        }
        bool grew = false;
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
            const int pair = dq * kOwn + x, head = pair / 2, slot = sg + pair % 2 * 8;
            if (!(mask >> slot & 1)) mine[x] = kNegInf;
            if (scores && head < rows) scores[head * score_pitch + slot] = mine[x];
            grew |= mine[x] > m[x / 2] + kSlack;
        }
        if (__any_sync(0xffffffffu, grew)) {
            float shrink[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                float v = mine[2 * i < kOwn ? 2 * i : 0];
                if (kOwn > 1) v = fmaxf(v, mine[2 * i + 1 < kOwn ? 2 * i + 1 : 0]);
                else v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                v = fmaxf(v, m[i]);
                shrink[i] = m[i] == kNegInf ? 0.0f : exp2f(m[i] - v);
                m[i] = v;
                l[i] *= shrink[i];
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                // Head h's pairs 2 h and 2 h + 1 belong to lane dq = 2 h / kOwn.
                const float f = __shfl_sync(0xffffffffu, shrink[kOwn > 1 ? h % kMine : 0], 2 * h / kOwn);
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[h][c][e] *= f;
            }
        }
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
            const int pair = dq * kOwn + x;
            const float w = exp2f(mine[x] - (m[x / 2] == kNegInf ? 0.0f : m[x / 2]));
            l[x / 2] += w;
            prob[(sg + pair % 2 * 8) * H + pair / 2] = w;
        }
        __syncwarp();
#pragma unroll 4
        for (int r = 0; r < 16; ++r) {
            float w[H];
#pragma unroll
            for (int h = 0; h < H; h += H == 2 ? 2 : 4) {
                if (H == 2) {
                    const float2 u = *reinterpret_cast<const float2 *>(prob + r * H);
                    w[0] = u.x;
                    w[1] = u.y;
                } else {
                    const float4 u = *reinterpret_cast<const float4 *>(prob + r * H + h);
                    w[h] = u.x;
                    w[h + 1] = u.y;
                    w[(h + 2) % H] = u.z;
                    w[(h + 3) % H] = u.w;
                }
            }
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int d = lane * 4 + c * 128;
                if (d >= D) continue;
                const float4 v = *reinterpret_cast<const float4 *>(v_rows + r * v_pitch(D) + d * 4);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    o[h][c][0] = fmaf(w[h], v.x, o[h][c][0]);
                    o[h][c][1] = fmaf(w[h], v.y, o[h][c][1]);
                    o[h][c][2] = fmaf(w[h], v.z, o[h][c][2]);
                    o[h][c][3] = fmaf(w[h], v.w, o[h][c][3]);
                }
            }
        }
        __syncwarp();
    }

    __device__ __forceinline__ void put(float *red_m, float *red_l, float *to, int pitch, int D) {
        const int lane = threadIdx.x % 32, sg = lane / 4, dq = lane % 4;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            float v = l[i];
            if (kOwn == 1) v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int head = dq * kOwn / 2 + i;
            if (sg == 0 && (kOwn > 1 || dq % 2 == 0)) {
                red_m[head] = m[i];
                red_l[head] = v;
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                if (lane * 4 + c * 128 < D)
                    *reinterpret_cast<float4 *>(to + h * pitch + lane * 4 + c * 128) =
                        make_float4(o[h][c][0], o[h][c][1], o[h][c][2], o[h][c][3]);
    }
};

template <typename C> inline size_t stage_bytes(int D) {
    return (size_t)16 * (C::k_pitch(D) + C::v_pitch(D));
}
template <typename C> inline size_t smem_bytes(int D, int B) {
    return (size_t)C::Shape::kWarps * C::Shape::kStages * stage_bytes<C>(D) + C::kSharedBytes + 8 * (size_t)B;
}

template <typename C>
__global__ void __launch_bounds__(32 * C::Shape::kWarps, C::Shape::kPerSm) attention_kernel(AttnParams p) {
    typedef typename C::Element T;
    constexpr int kWarps = C::Shape::kWarps, kThreads = 32 * kWarps, kTile = 16 * kWarps;
    constexpr int S = C::Shape::kStages, HN = C::kHeads, kD = C::kD;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t slot_masks[kWarps][S];
    __shared__ float red_m[kWarps][HN], red_l[kWarps][HN];
    __shared__ int warp_sum[kWarps];
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int D = kD ? kD : p.D;
    const int k_pitch = C::k_pitch(D), v_pitch = C::v_pitch(D), stage_bytes = 16 * (k_pitch + v_pitch);
    unsigned char *ring = smem + (size_t)warp * S * stage_bytes;
    unsigned char *shared = smem + (size_t)kWarps * S * stage_bytes;
    int *prefix = reinterpret_cast<int *>(shared + C::kSharedBytes);                  // [B]
    int *ntok = prefix + p.B;                                                         // [B]
    const bool with_new = p.k_new != nullptr;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // Entries and tiles before each sequence (of one head set), and all of them.
    auto lo_of = [&](int n) { return first_slot(p, n); };
    auto tiles_of = [&](int n) { return unit_tiles<kTile>(p, n); };
    int total;
    const int sets = (p.G + HN - 1) / HN, Hu = p.Hkv * sets;
    {
        const int per = (p.B + kThreads - 1) / kThreads, b0 = min(t * per, p.B),
                  b1 = min(b0 + per, p.B);
        int sum = 0, len;
        for (int b = b0; b < b1; ++b) {
            const int n = tokens_of(p.cache, b, with_new, &len);
            // The sign says whether the last token is the new one.
            ntok[b] = with_new && n > len && len >= 0 ? -n : n;
            sum += 1 + tiles_of(n);
        }
        __syncwarp();
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
            base += 1 + tiles_of(abs(ntok[b]));
        }
        total = all * Hu;       // at most 2^31 - 1: a plan's limit
        __syncthreads();
    }
    // Chunks of equal size, or whole units that the blocks take in turns.
    const int chunk = (total + gridDim.x - 1) / gridDim.x;
    if (p.whole_units ? (int)blockIdx.x >= p.B * Hu : (int)blockIdx.x * (int64_t)chunk >= total) return;

    auto enter = [&](Walk &w) {
        w.n = abs(ntok[w.b]);
        w.lo = lo_of(w.n);
        w.first = w.lo / kTile * kTile;
        w.tiles = tiles_of(w.n);
    };
    // The next segment of the walk: the tiles of one unit in the chunk.  False at the end.
    auto next_segment = [&](Walk &w) {
        if (p.whole_units) {
            const int u = (int)blockIdx.x + w.count * (int)gridDim.x;
            if (u >= p.B * Hu) return false;
            ++w.count;
            w.b = u / Hu;
            w.hv = u - w.b * Hu;
            enter(w);
            w.tile = 0;
            w.left = w.tiles;
            return true;
        }
        for (;;) {
            if (w.x >= w.x1) return false;
            if (w.x >= w.unit + 1 + w.tiles) {
                w.unit += 1 + w.tiles;
                if (++w.hv == Hu) {
                    w.hv = 0;
                    ++w.b;
                    enter(w);
                }
            }
            const int from = max(w.x, w.unit + 1), to = min(w.x1, w.unit + 1 + w.tiles);
            w.x = max(to, w.x + 1);
            if (from < to) {
                ++w.count;
                w.tile = from - (w.unit + 1);
                w.left = to - from;
                return true;
            }
        }
    };
    Walk use;
    use.left = use.count = 0;
    if (!p.whole_units) {
        use.x = blockIdx.x * chunk;
        use.x1 = min(total, use.x + chunk);
        const int q = use.x / Hu;
        int lo = 0, hi = p.B - 1;        // the last sequence with prefix <= q
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (prefix[mid] <= q) lo = mid; else hi = mid - 1;
        }
        use.b = lo;
        enter(use);
        use.hv = (use.x - prefix[lo] * Hu) / (use.tiles + 1);
        use.unit = prefix[lo] * Hu + use.hv * (use.tiles + 1);
    }

    // The producer side: kLanes lanes copy a row, 16 bytes each, kRows rows at a time.
    constexpr int kChunk = 16 / sizeof(T), kLanes = C::kMax / kChunk < 32 ? C::kMax / kChunk : 32;
    constexpr int kRows = 32 / kLanes, kRounds = 16 / kRows, kAcross = (C::kMax / kChunk + 31) / 32;
    Walk in = use;
    const bool more = next_segment(in);
    int ahead = 0, in_slot = 0;         // stages under way, and the next one to fill
    const int row0 = lane / kLanes, col = lane % kLanes;
    const bool copies = row0 < kRows && col * kChunk < D;
    // With pages of whole sixteens a warp's slots lie in one page.
    const bool one_page = p.cache.page % 16 == 0;
    // Offsets of rows in the pages, in sixteens of elements: a plan's pages have fewer than 2^32.
    const uint32_t page16 = (uint32_t)(p.cache.page_stride / 16), head16 = (uint32_t)(p.cache.head_stride / 16),
                   row16 = (uint32_t)(p.cache.row_stride / 16);
    const T *const k_col = static_cast<const T *>(p.k) + col * kChunk;
    const T *const v_col = static_cast<const T *>(p.v) + col * kChunk;
    const T *const k_lane = k_col + row0 * p.cache.row_stride, *const v_lane = v_col + row0 * p.cache.row_stride;
    const int64_t row_step = kRows * p.cache.row_stride;
    const uint32_t k_dst = ptx::smem_u32(ring) + row0 * k_pitch + col * 16;
    const uint32_t v_dst = ptx::smem_u32(ring) + 16 * k_pitch + row0 * v_pitch + col * 16;
    // Page numbers, fetched before they are wanted: one for each of 32 tiles where a warp's slots
    // lie in one page (lane i has tile pages_from + i's), else those of the next tile's slots.
    int pages = 0, pages_from = 0;
    auto page_index = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.cache.page; };
    auto fetch_pages = [&]() {
        const int j0 = in.first + in.tile * kTile + warp * 16;
        const int j = one_page ? j0 + lane * kTile : j0 + (lane & 15);
        pages_from = in.tile;
        // A warp's sixteen slots may begin before the window or end past the last token.
        const bool wanted = one_page ? j + 15 >= in.lo && j < in.n : j >= in.lo && j < in.n;
        pages = wanted ? __ldg(p.cache.tables + (int64_t)in.b * p.cache.table_pitch + page_index(j)) : -1;
    };
    // Fills a stage with the next tile, if the walk has one.
    auto issue = [&]() {
        if (in.left == 0) return;
        {
            const int j0 = in.first + in.tile * kTile + warp * 16, j = j0 + (lane & 15);
            const int hk = sets == 1 ? in.hv : in.hv / sets;
            const int page_no = one_page ? __shfl_sync(0xffffffffu, pages, in.tile - pages_from) : pages;
            const bool inside = j >= in.lo && j < in.n;
            const bool ok = inside && (unsigned)page_no < (unsigned)p.cache.num_pages;
            const unsigned mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            const uint32_t off = page_no * page16 + hk * head16 + (j - page_index(j) * p.cache.page) * row16;
            if (lane == 0) slot_masks[warp][in_slot] = mask;
            if (inside && !ok)
                atomicOr(p.cache.status, kStatusBadPage);
            const uint32_t kd = k_dst + in_slot * stage_bytes, vd = v_dst + in_slot * stage_bytes;
            const int newest = ntok[in.b];       // -n where slot n - 1 is the new token's
            const bool plain = mask == 0xffffu && !(newest < 0 && -newest - 1 < j0 + 16);
            if (plain && one_page) {
                const int64_t first = (int64_t)__shfl_sync(0xffffffffu, off, 0) * 16;
                const T *ks = k_lane + first, *vs = v_lane + first;
                if (kD && kAcross == 1 && p.cache.row_stride == kD) {
                    // Rows one behind the other: every offset is a constant.
#pragma unroll
                    for (int i = 0; copies && i < kRounds; ++i) {
                        copy16(kd + i * kRows * k_pitch, ks + i * kRows * kD, true);
                        copy16(vd + i * kRows * v_pitch, vs + i * kRows * kD, true);
                    }
                } else if (copies) {
#pragma unroll
                    for (int i = 0; i < kRounds; ++i) {
#pragma unroll
                        for (int x = 0; x < kAcross; ++x) {
                            if (x > 0 && (col + 32 * x) * kChunk >= D) break;
                            copy16(kd + i * kRows * k_pitch + x * 512, ks + x * 32 * kChunk, true);
                            copy16(vd + i * kRows * v_pitch + x * 512, vs + x * 32 * kChunk, true);
                        }
                        ks += row_step;
                        vs += row_step;
                    }
                }
            } else if (plain) {
                // Rows of several pages, all of them wanted.  (fp32, 47 sequences of 4 heads of 80, pages of
                // 8: 52 us, and 63 the general way below.)
#pragma unroll 4
                for (int i = 0; i < kRounds; ++i) {
                    const int64_t o = (int64_t)__shfl_sync(0xffffffffu, off, (i * kRows + row0) & 15) * 16;
#pragma unroll
                    for (int x = 0; x < kAcross; ++x) {
                        if (!copies || (x > 0 && (col + 32 * x) * kChunk >= D)) continue;
                        copy16(kd + i * kRows * k_pitch + x * 512, k_col + o + x * 32 * kChunk, true);
                        copy16(vd + i * kRows * v_pitch + x * 512, v_col + o + x * 32 * kChunk, true);
                    }
                }
            } else {
                const int64_t at_new = in.b * p.kv_stride + (int64_t)hk * D;
                const T *const k_new = static_cast<const T *>(p.k_new) + at_new;
                const T *const v_new = static_cast<const T *>(p.v_new) + at_new;
#pragma unroll 4
                for (int i = 0; i < kRounds; ++i) {
                    const int row = (i * kRows + row0) & 15;
                    const int64_t o = (int64_t)__shfl_sync(0xffffffffu, off, row) * 16;
                    const bool on = mask >> row & 1;
                    // The new token's row comes from the arguments.
                    const bool fresh = newest == -(j0 + row + 1);
                    const T *ks = fresh ? k_new : static_cast<const T *>(p.k) + o;
                    const T *vs = fresh ? v_new : static_cast<const T *>(p.v) + o;
                    // Hidden slots are filled with zeros: no probability is given to them, and
                    // what V holds there must be finite.  (The address is not read.)
#pragma unroll
                    for (int x = 0; x < kAcross; ++x) {
                        const int c = (col + 32 * x) * kChunk;
                        if (!copies || c >= D) continue;
                        copy16(kd + i * kRows * k_pitch + x * 512, on ? ks + c : p.k, on);
                        copy16(vd + i * kRows * v_pitch + x * 512, on ? vs + c : p.v, on);
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++ahead;
        if (++in_slot == S) in_slot = 0;
        ++in.tile;
        if (--in.left == 0) {
            if (next_segment(in)) fetch_pages();
        } else if (!one_page || in.tile - pages_from == 32) {
            fetch_pages();
        }
    };
    if (more) fetch_pages();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) issue();
    int slot = 0;
    C heads;
    auto load_queries = [&]() {
        const int hk = use.hv / sets, set = use.hv % sets, first = hk * p.G + set * HN;
        heads.load_queries(static_cast<const T *>(p.q) + use.b * p.q_stride + first * D, p.G - set * HN, D,
                           shared);
    };
    bool go = next_segment(use);
    if (go) load_queries();
    if (C::kSharedQueries) __syncthreads();
    while (go) {
        // One unit's share of a chunk.
        const int hk = use.hv / sets, set = use.hv % sets;
        const int rows = min(HN, p.G - set * HN);
        const int64_t h0 = (int64_t)use.b * p.Hq + (int64_t)hk * p.G + set * HN;   // first query head
        const int steps = use.left;
        const int unit_b = use.b;
        const bool whole = use.tile == 0 && steps == use.tiles;
        const int part = blockIdx.x * 2 + (use.count == 1 ? 0 : 1);
        // The slot that this unit puts in the cache, once for a KV head.
        const int new_slot = ntok[use.b] < 0 && set == 0 ? use.n - 1 : -1;
        const int j_first = use.first + use.tile * kTile + warp * 16;
        heads.reset();
        for (int step = 0; step < steps; ++step) {
            if (ahead >= S - 1)
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            else
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            const uint32_t mask = slot_masks[warp][slot];
            --ahead;
            issue();
            const unsigned char *slot_base = ring + slot * stage_bytes;
            if (++slot == S) slot = 0;
            if (new_slot >= 0) {
                // The new token's row goes on to the cache.
                const int row = new_slot - (j_first + step * kTile);
                if (row >= 0 && row < 16 && (mask >> row & 1)) {
                    const int pg = p.cache.tables[(int64_t)unit_b * p.cache.table_pitch + page_index(new_slot)];
                    const int64_t to = pg * p.cache.page_stride + hk * p.cache.head_stride +
                                       (new_slot - page_index(new_slot) * p.cache.page) * p.cache.row_stride;
                    const uint4 *kf = reinterpret_cast<const uint4 *>(slot_base + row * k_pitch);
                    const uint4 *vf = reinterpret_cast<const uint4 *>(slot_base + 16 * k_pitch + row * v_pitch);
                    for (int c = lane; c < D / kChunk; c += 32) {
                        reinterpret_cast<uint4 *>(static_cast<T *>(p.k) + to)[c] = kf[c];
                        reinterpret_cast<uint4 *>(static_cast<T *>(p.v) + to)[c] = vf[c];
                    }
                }
            }
            if (mask == 0 && !p.scores) continue;
            // The score rows cover whole tiles.
            heads.step(slot_base, slot_base + 16 * k_pitch, mask, D, p.scale_log2, rows,
                       p.scores ? p.scores + h0 * p.score_pitch + j_first + step * kTile : nullptr,
                       p.score_pitch, shared);
        }

        // Join the warps, through the stage that each has just used: it is filled again in the
        // next step at the earliest, and holds [HN][D + 4] fp32.
        const int used = (slot == 0 ? S : slot) - 1, join_pitch = D + 4;
        __syncwarp();
        heads.put(red_m[warp], red_l[warp], reinterpret_cast<float *>(ring + used * stage_bytes), join_pitch, D);
        __syncthreads();
        // The next unit's queries come in meanwhile.
        go = next_segment(use);
        if (go) load_queries();
        constexpr int kQuads = C::kMax / 4;
#pragma unroll
        for (int x0 = 0; x0 < HN * kQuads; x0 += kThreads) {
            const int head = (x0 + t) / kQuads, d = (x0 + t) % kQuads * 4;
            if (head >= rows || d >= D) continue;
            float top = kNegInf, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][head]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = red_m[w][head] == kNegInf ? 0.0f : pow2(red_m[w][head] - top);
                const float4 u = *reinterpret_cast<const float4 *>(
                    smem + (size_t)(w * S + used) * stage_bytes + (head * join_pitch + d) * 4);
                sum = fmaf(red_l[w][head], f, sum);
                v.x = fmaf(u.x, f, v.x);
                v.y = fmaf(u.y, f, v.y);
                v.z = fmaf(u.z, f, v.z);
                v.w = fmaf(u.w, f, v.w);
            }
            if (whole) {
                const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
                // (A head without weight is 0 whatever V holds: 0 times an infinity would be NaN.)
                if (sum == 0.0f) v = make_float4(0.f, 0.f, 0.f, 0.f);
                store4(static_cast<T *>(p.out) + (h0 + head) * D + d, v.x * r, v.y * r, v.z * r, v.w * r);
                if (p.scores && d == 0) p.stats[h0 + head] = make_float2(top, sum);
            } else {
                const int64_t row = (int64_t)part * p.part_rows + head;
                *reinterpret_cast<float4 *>(p.part_o + row * D + d) = v;
                if (d == 0) p.part_ml[row] = make_float2(top, sum);
            }
        }
        __syncthreads();
    }
}


// The second kernel: joins the parts of the units that several chunks share, in chunk order.
// kRowWarps warps take one query head, each a run of its parts kDepth at a time.  What it reads
// is in L2; its time is the launch, which overlaps the first kernel's end, and one or two trips to
// L2.
constexpr int kJoinWarps = 8;
template <typename T, int hn, int kTile, int N, int kRowWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(AttnParams p, int grid) {
    constexpr int kDepth = 16 / N, kRows = kJoinWarps / kRowWarps;
    __shared__ float2 ml[kJoinWarps];
    __shared__ __align__(16) float outs[kJoinWarps][256];
    const int t = threadIdx.x, warp = t / 32, lane = t % 32, sub = warp % kRowWarps;
    const int64_t row_no = (int64_t)blockIdx.x * kRows + warp / kRowWarps;    // b * Hq + head
    // A block's heads may belong to two sequences: each warp sums up for its own.
    const bool on = row_no < (int64_t)p.B * p.Hq;
    const int b = on ? (int)(row_no / p.Hq) : p.B - 1, h = on ? (int)(row_no % p.Hq) : 0;
    const int sets = (p.G + hn - 1) / hn, Hu = p.Hkv * sets;
    // The lengths are read before the wait below: attention_kernel only reads them too, and has waited for
    // all kernels before it when it lets this one start.
    int before = 0, all = 0, mine = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int tiles = unit_tiles<kTile>(p, token_count(p.cache, i, p.k_new != nullptr));
        all += 1 + tiles;
        if (i < b) before += 1 + tiles;
        if (i == b) mine = tiles;
    }
    __syncwarp();
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    const int tiles = __reduce_add_sync(0xffffffffu, mine);
    const int total = all * Hu, chunk = (total + grid - 1) / grid;
    const int hk = h / p.G, g = h % p.G, hv = hk * sets + g / hn, row = g % hn;
    const int unit = before * Hu + hv * (tiles + 1);
    const int c0 = (unit + 1) / chunk, parts = on ? (unit + tiles) / chunk - c0 + 1 : 1;
    // The first part is its chunk's first unless the chunk has tiles of an earlier unit.
    const int head = c0 * 2 + (c0 * chunk >= unit ? 0 : 1);
    ptx::griddep_wait();
    if (kRowWarps == kJoinWarps && parts == 1) return;
    // This warp's run of the parts.
    const int run = (parts + kRowWarps - 1) / kRowWarps, from = min(sub * run, parts),
              to = parts == 1 ? from : min(from + run, parts);
    float M = kNegInf, L = 0.0f;
    float4 v[N];                     // columns lane * 4 (and, past 128 of them, 128 further)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int d = lane * 4;
    for (int c = from; c < to; c += kDepth) {
        // Past the end the last part is read again, for nothing: loads behind a condition would
        // wait for one another.
        float2 s[kDepth];
        float4 u[N][kDepth];
#pragma unroll
        for (int y = 0; y < kDepth; ++y) {
            const int at = min(c + y, to - 1);
            const int64_t id = (int64_t)(at == 0 ? head : (c0 + at) * 2) * p.part_rows + row;
            s[y] = __ldcg(p.part_ml + id);
#pragma unroll
            for (int i = 0; i < N; ++i)
                u[i][y] = __ldcg(reinterpret_cast<const float4 *>(
                    p.part_o + id * p.D + min(d + i * 128, p.D - 4)));
        }
        float M2 = M;
#pragma unroll
        for (int y = 0; y < kDepth; ++y) {
            if (c + y >= to) {
                // (Infinite outputs would make 0 times them NaN.)
                s[y] = make_float2(kNegInf, 0.0f);
#pragma unroll
                for (int i = 0; i < N; ++i) u[i][y] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            M2 = fmaxf(M2, s[y].x);
        }
        const float shrink = M == kNegInf ? 0.0f : pow2(M - M2);
        M = M2;
        L *= shrink;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i].x *= shrink;
            v[i].y *= shrink;
            v[i].z *= shrink;
            v[i].w *= shrink;
        }
#pragma unroll
        for (int y = 0; y < kDepth; ++y) {
            const float f = s[y].x == kNegInf ? 0.0f : pow2(s[y].x - M);
            L = fmaf(s[y].y, f, L);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i].x = fmaf(u[i][y].x, f, v[i].x);
                v[i].y = fmaf(u[i][y].y, f, v[i].y);
                v[i].z = fmaf(u[i][y].z, f, v[i].z);
                v[i].w = fmaf(u[i][y].w, f, v[i].w);
            }
        }
    }
    if (lane == 0) ml[warp] = make_float2(M, L);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (d + i * 128 < p.D) *reinterpret_cast<float4 *>(&outs[warp][d + i * 128]) = v[i];
    __syncthreads();
    if (sub != 0 || parts == 1) return;
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, ml[warp + w].x);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        const float f = ml[warp + w].x == kNegInf ? 0.0f : pow2(ml[warp + w].x - top);
        sum = fmaf(ml[warp + w].y, f, sum);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (d + i * 128 >= p.D) continue;
            const float4 u = *reinterpret_cast<const float4 *>(&outs[warp + w][d + i * 128]);
            v[i].x = fmaf(u.x, f, v[i].x);
            v[i].y = fmaf(u.y, f, v[i].y);
            v[i].z = fmaf(u.z, f, v[i].z);
            v[i].w = fmaf(u.w, f, v[i].w);
        }
    }
    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (sum == 0.0f) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d + i * 128 < p.D)
            store4(static_cast<T *>(p.out) + row_no * p.D + d + i * 128, v[i].x * r, v[i].y * r, v[i].z * r,
                   v[i].w * r);
    }
    if (p.scores && lane == 0) p.stats[row_no] = make_float2(top, sum);
}

}  // namespace attn
}  // namespace ctr
