// chunk_tc.cuh -- attention of a chunk of new tokens over a paged 16-bit cache, on the tensor cores.
//
// Two products a tile of 128 rows by NT slots, S = Q K^T and O += P V, 4 D operations a score against
// one exponential, a maximum, a sum and a rounding: with many rows the tensor pipe bounds it, with few
// the cache's bytes.  A block has two tiles of 128 rows on the same slots (one where D > 128), so that
// K and V are read from L2 once for 256 rows and the tensor pipe works on one tile's products while
// the other's softmax runs:
//   warps 0-3, 4-7  the softmax of each tile, a thread a row: S from TMEM, P to TMEM over it;
//   warps 8-11      copy K and V slots, wherever their pages are, and Q rows into shared memory, a
//                   ring of stages of one K or V tile each (cp.async: 16 bytes from any page, zeros
//                   for slots that are not there);
//   warp 12         issues tcgen05.mma: per tile of slots PV0, QK0 of the next tile, PV1, QK1;
//   warp 13         describes the block's segments (chunk_schedule.cuh) ahead of the others.
// P stays in TMEM as the first operand of PV (half the shared-memory reads of one from there),
// and V is read as it lies, [slots][columns], as a column-major operand.  With one tile of rows the
// two S buffers alternate instead.
//
// 512 tokens on 65531 cached ones, 32/8 heads of 128, bf16: 485 to 494 us (1.13 PFLOP/s, 57% of cuBLAS's measured
// rate) through the API with inputs in turn, 433 to 447 in a captured graph of one call again and again.  Its K and V,
// 270 MB, do not fit the L2, and the row tiles of a head walk them at different times: 2.16 GB come from memory.  Of
// the 433, without the softmax 343, the products alone 307.  8192 tokens: 493 us.  In graphs, 2048 tokens on
// 16384: 409 us for heads of 64 (the softmax bounds it), 453 for 128, 985 for 256.  16 single tokens on 8192 slots
// each: 98 us (5.5 TB/s).  4 tokens on 125: 10 to 11 us.
//
// Softmax: powers of two of a score's distance to the row's base, which follows the running maximum only when
// that exceeds it by kSlack, because then O has to be rescaled in TMEM, which the tensor pipe waits
// for.  Rows are independent of one another to the last bit.
//
// Rounding: scores, statistics and O are fp32; P is rounded once to the type (half the operations of two
// terms; the error is that of one rounding of the output, and smaller where weights are many), the
// sum is that of the unrounded ones.  fp16 has no exponents to spare below 2^-24: its P is lifted
// by 2^13 and its slack is 2^2, so that weights keep eleven bits down to 2^-27 of the largest.
#pragma once

#include <algorithm>
#include <type_traits>

#include "chunk_device.cuh"
#include "chunk_join.cuh"

namespace ctr {
namespace chunk {

template <typename T> struct Half;
template <> struct Half<__nv_bfloat16> {
    static constexpr float kLift = 0.0f, kSlack = 8.0f;
    static constexpr uint32_t kFormat = ptx::kFmtBF16, kExponent = 0x7f80u;
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return ptx::bf16x2_rn(a, b); }
    // (bf16 has fp32's exponents: nothing to hold up.)
    static __device__ __forceinline__ uint32_t hold_up(uint32_t v) { return v; }
};
template <> struct Half<__half> {
    static constexpr float kLift = 13.0f, kSlack = 2.0f;
    static constexpr uint32_t kFormat = ptx::kFmtF16, kExponent = 0x7c00u;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
    // At least 2^-24 (2^-37 of the largest), so that an infinite V stays infinite.
    static __device__ __forceinline__ uint32_t hold_up(uint32_t v) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x00010001u));
        return r;
    }
};

// Sizes by the largest head size.
template <int DP> struct Sizes {
    static constexpr int kTiles = DP <= 128 ? 2 : 1;           // of 128 rows
    static constexpr int kRows = 128 * kTiles, kSlots = DP <= 128 ? 128 : 64;
    static constexpr int kPanels = DP / 64;                    // of 128 bytes of every row
    static constexpr int kQPanel = 128 * 128, kPanel = kSlots * 128;
    static constexpr int kStage = kPanels * kPanel;
    static constexpr int kStages = DP <= 64 ? 8 : 5;
    static constexpr int kQ = kTiles * kPanels * kQPanel;
    static constexpr int kSmem = 1024 + kQ + kStages * kStage;
    // TMEM columns.
    static constexpr int kS = 0, kO = 2 * kSlots, kOPitch = DP;
    static_assert(kO + kTiles * kOPitch <= 512, "TMEM");
};

constexpr int kThreads = 512, kCopyWarp = 8, kMmaWarp = 12, kScheduleWarp = 13;
constexpr int kRing = 8;                                        // tiles whose visible slots are kept
constexpr int kSegments = 8;                                    // segments that the schedule is ahead
constexpr int kSoftmaxRegs = 192, kCopyRegs = 72, kMmaRegs = 56;  // 256 * 192 + 128 (72 + 56) = 512 * 128

// What the roles know of a segment: the unit (as in Unit) and its tiles [t0, t1); none: the end.
struct Segment {
    Sequence s;
    int b, hk, m, r0, rows, lo, hi, lo_last, hi_first, first;
    int t0, t1;
    int part, begins, parts; // as in Walk
    int taint;               // values that are no numbers were taken out of V
};

template <bool kPolled> struct Shared {
    // Whoever waits at a barrier waits for each of its phases in turn, or knows by what it has seen
    // that the earlier ones are over: a wait tells only odd phases from even ones.  So where one tile of
    // rows uses both S buffers, the second has barriers of its own ([2]).
    uint64_t kv_full[8], kv_empty[8], q_full, q_empty, s_full[3], p_full[3], o_full[2], drained;
    uint64_t segment_full[kSegments], segment_empty[kSegments];
    Segment segments[kSegments];
    uint32_t visible[kRing][4];
    uint32_t tmem;
    volatile int abort;
    uint64_t copied;
};

// Bounded; every lane asks, and the answer is a vote: behind a branch the compiler takes the warp for
// divided, and its products and TMEM accesses for many (which took twice the time).
// try_wait sleeps for longer than any healthy wait takes, so that another limit than the default is kept by asking
// test_wait instead: by a kernel of its own (kPolled), because a choice at every wait took 5 to 12% of the time and
// a limit that is no constant 2.
template <bool kPolled>
__device__ __forceinline__ bool tested(const ChunkParams &p, Shared<kPolled> &sh, uint64_t *bar, uint32_t parity) {
    if constexpr (kPolled) {
        const uint64_t start = ptx::globaltimer_ns();
        bool there;
        while (!(there = ptx::mbar_test_wait(bar, parity)) && !sh.abort &&
               ptx::globaltimer_ns() - start < p.wait_limit_ns) {
        }
        return __all_sync(0xffffffffu, there);
    } else {
        return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity));
    }
}
template <bool kPolled>
__device__ __forceinline__ bool wait(const ChunkParams &p, Shared<kPolled> &sh, uint64_t *bar, uint32_t parity) {
    if (tested(p, sh, bar, parity)) return true;
    return !kPolled && ptx::mbar_wait_warp(bar, parity, kChunkWaitLimitNs, &sh.abort);
}
template <bool kPolled> __device__ __forceinline__ void give_up(Shared<kPolled> &sh, const ChunkParams &p) {
    sh.abort = 1;
    if (threadIdx.x % 32 == 0) atomicOr(p.cache.status, kStatusTimeout);
}

// The next segment's description, or null at the end (ok stays) or when a wait fails; and done with one.
template <bool kPolled>
__device__ __forceinline__ Segment *next_segment(const ChunkParams &p, Shared<kPolled> &sh, int no, bool &ok) {
    ok = wait(p, sh, &sh.segment_full[no % kSegments], no / kSegments & 1);
    Segment *s = &sh.segments[no % kSegments];
    return ok && s->t1 > s->t0 ? s : nullptr;
}
template <bool kPolled> __device__ __forceinline__ void segment_done(Shared<kPolled> &sh, int no) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) ptx::mbar_arrive(&sh.segment_empty[no % kSegments]);
    __syncwarp();
}

// Describes the block's segments, ahead of the roles that work on them.
template <int MT, int NT, bool kPolled>
__device__ __forceinline__ bool schedule(const ChunkParams &p, Shared<kPolled> &sh, const int64_t *costs) {
    Walk<MT, NT> walk;
    walk.start(p, find_start<MT, NT>(p, costs));
    for (int no = 0;; ++no) {
        const bool more = walk.next(p);
        if (!wait(p, sh, &sh.segment_empty[no % kSegments], (no / kSegments & 1) ^ 1)) return false;
        if (threadIdx.x % 32 == 0) {
            const Unit<MT, NT> &u = walk.u;
            Segment &s = sh.segments[no % kSegments];
            s.t0 = s.t1 = 0;
            if (more) {
                s.s = u.s;
                s.b = u.b;
                s.hk = u.hk;
                s.m = u.m;
                s.r0 = u.r0;
                s.rows = u.rows;
                s.lo = u.lo;
                s.hi = u.hi;
                s.lo_last = u.lo_last;
                s.hi_first = u.hi_first;
                s.first = u.first;
                s.t0 = walk.t0;
                s.t1 = walk.t1;
                s.part = walk.part;
                s.begins = walk.begins;
                s.parts = walk.parts();
                s.taint = 0;
            }
            ptx::mbar_arrive(&sh.segment_full[no % kSegments]);
        }
        __syncwarp();
        if (!more) return true;
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Products whose operands lie `kA` and `kB` sixteen-byte units behind descriptors that differ in their lower
// words only (the upper one: eight rows of 128 bytes a group, 128-byte swizzle): the additions belong to the
// product, where the compiler does not keep a descriptor for each in registers.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
template <int kA, int kB>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "add.u32 x, %1, %6;\n\tadd.u32 y, %2, %7;\n\t"
                 "mov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHigh), "n"(kA), "n"(kB)
                 : "memory");
}
// The first operand in TMEM.
template <int kA, int kB>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "add.u32 x, %1, %6;\n\tadd.u32 y, %2, %7;\n\t"
                 "mov.b64 b, {y, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHigh), "n"(kA), "n"(kB)
                 : "memory");
}
// The lower word for rows of K-major panels, and for a [k][n] operand of panels of 64 columns, `panel` bytes
// apart, whose rows are k.
__device__ __forceinline__ uint32_t desc_k(uint32_t smem_addr) { return (smem_addr >> 4 & 0x3fff) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t smem_addr, uint32_t panel) {
    return (smem_addr >> 4 & 0x3fff) | panel >> 4 << 16;
}
constexpr uint32_t kTransposeB = 1u << 16;

// f(0), f(1), ... with constants.
template <int kN, int kI = 0, typename F> __device__ __forceinline__ void each(F &&f) {
    if constexpr (kI < kN) {
        f(std::integral_constant<int, kI>());
        each<kN, kI + 1>(f);
    }
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                   "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
                   "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                   "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                   "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// (Two fp32 operations an instruction, as pair() and fma2().)
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The slots [j0 + 32 w, + 32) that lie in [lo, hi), as bits.
__device__ __forceinline__ uint32_t range_bits(int j, int lo, int hi) {
    const int a = min(max(lo - j, 0), 32), b = min(max(hi - j, 0), 32);
    return (uint32_t)((1ull << b) - (1ull << min(a, b)));
}

// Takes values that are no numbers out of this thread's part of a V stage (see taint); whether there
// were any.
template <typename T, int DP> __device__ __noinline__ bool take_out(uint32_t stage, int D) {
    typedef Sizes<DP> Z;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kCopyWarp;
    bool found = false;
    for (int panel = 0; panel * 64 < D; ++panel) {
        if (panel * 64 + lane % 8 * 8 >= D) continue;
        for (int r = lane / 8; r < Z::kSlots / 4; r += 4) {
            const int row = warp * (Z::kSlots / 4) + r;
            const uint32_t at = stage + panel * Z::kPanel + row * 128 + ((lane ^ row) & 7) * 16;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr uint32_t kE = Half<T>::kExponent;
                if ((v[i] & kE) == kE) v[i] &= 0xffff0000u, bad = true;
                if ((v[i] >> 16 & kE) == kE) v[i] &= 0x0000ffffu, bad = true;
            }
            if (bad) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
                             "r"(v[2]), "r"(v[3]) : "memory");
                found = true;
            }
        }
    }
    return found;
}

// ------------------------------------------------------------------------------------------------
// Copies.  Each of the four warps has a quarter of a tile's slots: a lane looks one up, then eight
// lanes copy 128 bytes of one.
template <typename T, int DP, bool kPolled> struct Copier {
    typedef Sizes<DP> Z;
    const ChunkParams &p;
    Shared<kPolled> &sh;
    uint32_t q_smem, kv_smem;
    int items;
    int looked;              // the stage of a V tile that is still to be looked through, or -1,
    int looked_in;           // its segment,
    bool left;               // and whether that is done but for this

    // The barrier's phase ends when this thread's copies, and those of all others, have arrived.
    __device__ __forceinline__ void arrive(uint64_t *bar) {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
    }
    // Looks a V tile through (see taint) once its copies, all but the last kLater groups, have arrived.
    template <int kLater> __device__ __forceinline__ void look() {
        if (looked < 0) return;
        copy_wait<kLater>();
        if (take_out<T, DP>(kv_smem + looked * Z::kStage, p.D))
            sh.segments[looked_in % kSegments].taint = 1;
        __syncwarp();
        fence_async();
        ptx::mbar_arrive(&sh.kv_full[looked]);
        looked = -1;
        if (left) segment_done(sh, looked_in);
        left = false;
        __syncwarp();
    }
    // Waits for a phase; whoever completes it may be waiting for the tile that is to be looked through.
    __device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity) {
        if (tested(p, sh, bar, parity)) return true;
        look<0>();
        return wait(p, sh, bar, parity);
    }

    // kRows rows of a warp, panels of 128 bytes: lane l's row is at `from` + `mine` elements, if there is one.
    template <int kRows, int kPanel, int kUnroll, typename Offset>
    __device__ __forceinline__ void copy_rows(uint32_t dst, const T *from, Offset mine, bool on, int unit) {
        const int lane = threadIdx.x % 32, column = lane % 8 * 8;
        const unsigned there = __ballot_sync(0xffffffffu, on);
        const int D = p.D;
        const uint32_t to = dst + lane / 8 * 128 + ((lane ^ lane / 8) & 7) * 16;
        from += column;
#pragma unroll kUnroll
        for (int r0 = 0; r0 < kRows; r0 += 4) {
            const int r = r0 + lane / 8;
            const T *src = from + (int64_t)__shfl_sync(0xffffffffu, mine, r) * unit;
            const bool ok = there >> r & 1;
            // (The swizzle is the row's last three bits; every other step changes the third.)
            const uint32_t at = (to ^ (r0 % 8 ? 64 : 0)) + r0 * 128;
#pragma unroll
            for (int panel = 0; panel < Z::kPanels; ++panel)
                if (panel * 64 + column < D) copy16(at + panel * kPanel, src + panel * 64, ok);
        }
    }

    __device__ __forceinline__ bool run() {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kCopyWarp;
        constexpr int kOwn = Z::kSlots / 4;
        int tiles = 0;
        bool ok;
        items = 0;
        looked = -1;
        left = false;
        for (int no = 0;; ++no) {
            const Segment *const next = next_segment(p, sh, no, ok);
            if (!next) {
                look<0>();
                return ok;
            }
            const Segment &u = *next;
            const int t0 = u.t0, t1 = u.t1;
            for (int t = t0; t < t1; ++t, ++tiles) {
                const int j0 = (u.first + t) * Z::kSlots;
                const bool edge = is_edge(u, j0, Z::kSlots);
                const int64_t at = lane < kOwn ? cache_row(p.cache, p.page_shift, u, j0 + warp * kOwn + lane) : -1;
                const bool on = at >= 0;
                const uint32_t mine = on ? (uint32_t)(at >> 4) : 0u;
                const unsigned seen = __ballot_sync(0xffffffffu, on);
                // K, on the first tile Q, and V.
                for (int kv = 0; kv < 2; ++kv, ++items) {
                    const int stage = items % Z::kStages;
                    if (!wait_for(&sh.kv_empty[stage], (items / Z::kStages & 1) ^ 1)) return false;
                    copy_rows<kOwn, Z::kPanel, kOwn / 4>(kv_smem + stage * Z::kStage + warp * kOwn * 128,
                                               (const T *)(kv ? p.v : p.k), mine, on, 16);
                    copy_commit();
                    if (kv == 0) {
                        if (lane == 0) {
                            if (kOwn == 32) sh.visible[tiles % kRing][warp] = seen;
                            else reinterpret_cast<uint16_t *>(sh.visible[tiles % kRing])[warp] = (uint16_t)seen;
                            __threadfence_block();       // the arrival below is its copies', not its own
                        }
                        __syncwarp();
                        arrive(&sh.kv_full[stage]);
                        look<1>();
                        if (t == t0 && !queries(u, no)) return false;
                    } else if (edge) {
                        looked = stage;
                        looked_in = no;
                    } else {
                        arrive(&sh.kv_full[stage]);
                    }
                }
            }
            // The last tile is looked through behind the next segment's first copies.
            left = looked >= 0;
            if (!left) segment_done(sh, no);
        }
    }
    __device__ __forceinline__ bool queries(const Segment &u, int no) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kCopyWarp;
        if (!wait_for(&sh.q_empty, (no & 1) ^ 1)) return false;
#pragma unroll 1
        for (int tile = 0; tile < Z::kTiles; ++tile) {
            if (tile * 128 >= u.rows) break;
            const int r = tile * 128 + warp * 32 + lane;
            const bool on = r < u.rows;
            const int64_t mine = on ? query_offset(p, u, r) : 0;
            copy_rows<32, Z::kQPanel, 2>(q_smem + tile * Z::kPanels * Z::kQPanel + warp * 32 * 128, (const T *)p.q,
                                      mine, on, 1);
        }
        arrive(&sh.q_full);
        return true;
    }
};

// ------------------------------------------------------------------------------------------------
// Products.
template <typename T, int DP, bool kPolled> struct Multiplier {
    typedef Sizes<DP> Z;
    const ChunkParams &p;
    Shared<kPolled> &sh;
    uint32_t q_smem, kv_smem, tmem;

    // (One elected lane issues a tile's products in a row, their descriptors a constant apart.)
    __device__ __forceinline__ void scores(int tile, int buffer, int stage) {
        const uint32_t idesc = ptx::idesc_f32acc(Half<T>::kFormat, 128, Z::kSlots);
        const uint32_t q = desc_k(q_smem + tile * Z::kPanels * Z::kQPanel), k = desc_k(kv_smem + stage * Z::kStage);
        const uint32_t s = tmem + Z::kS + buffer * Z::kSlots;
        const int D = p.D;
        if (ptx::elect_one())
            each<DP / 16>([&](auto step) {
                constexpr int i = decltype(step)::value;
                if (i * 16 < D)
                    mma_ss<(i / 4 * Z::kQPanel + i % 4 * 32) / 16, (i / 4 * Z::kPanel + i % 4 * 32) / 16>(
                        s, q, k, idesc, i > 0);
            });
    }
    __device__ __forceinline__ void values(int tile, int buffer, int stage, bool first) {
        const uint32_t idesc = ptx::idesc_f32acc(Half<T>::kFormat, 128, p.D) | kTransposeB;
        const uint32_t v = desc_mn(kv_smem + stage * Z::kStage, Z::kPanel);
        const uint32_t o = tmem + Z::kO + tile * Z::kOPitch;
        const uint32_t w = tmem + Z::kS + buffer * Z::kSlots;
        if (ptx::elect_one())
            each<Z::kSlots / 16>([&](auto step) {
                constexpr int i = decltype(step)::value;
                mma_ts<i * 8, i * 2048 / 16>(o, w, v, idesc, i > 0 || !first);
            });
    }
    // The barrier's phase ends when the products issued so far do; the plain arrival orders what this
    // warp has seen before it for who waits there.
    __device__ __forceinline__ void commit(uint64_t *bar) {
        if (ptx::elect_one()) {
            ptx::mma_commit(bar);
            ptx::mbar_arrive(bar);
        }
    }
    __device__ __forceinline__ void release(uint64_t *bar) {
        if (ptx::elect_one()) ptx::mma_commit(bar);
    }
    // Waits for copies, whose writes the products then see.
    __device__ __forceinline__ bool arrived(uint64_t *bar, uint32_t parity) {
        const bool ok = wait(p, sh, bar, parity);
        fence_async();
        return ok;
    }
    __device__ __forceinline__ bool arrived(int item) {
        return arrived(&sh.kv_full[item % Z::kStages], item / Z::kStages & 1);
    }

    __device__ __forceinline__ bool run() {
        int items = 0, p_count[3] = {0, 0, 0};
        bool ok;
        for (int no = 0;; ++no) {
            const Segment *const u = next_segment(p, sh, no, ok);
            if (!u) return ok;
            const int n = u->t1 - u->t0;
            const bool dual = u->rows > 128;
            segment_done(sh, no);
            if (!arrived(&sh.q_full, no & 1) || !arrived(items)) return false;
            ptx::tc_fence_after();
            scores(0, 0, items % Z::kStages);
            commit(&sh.s_full[0]);
            if (dual) {
                scores(1, 1, items % Z::kStages);
                commit(&sh.s_full[1]);
            }
            release(&sh.kv_empty[items % Z::kStages]);
            if (n == 1) release(&sh.q_empty);
            for (int t = 0; t < n; ++t, items += 2) {
                const int v = (items + 1) % Z::kStages, k = (items + 2) % Z::kStages;
                const bool more = t + 1 < n;
                if (dual) {
                    if (!arrived(items + 1) || !wait(p, sh, &sh.p_full[0], p_count[0]++ & 1)) return false;
                    ptx::tc_fence_after();
                    values(0, 0, v, t == 0);
                    commit(&sh.o_full[0]);
                    if (more) {
                        if (!arrived(items + 2)) return false;
                        ptx::tc_fence_after();
                        scores(0, 0, k);
                        commit(&sh.s_full[0]);
                    }
                    if (!wait(p, sh, &sh.p_full[1], p_count[1]++ & 1)) return false;
                    ptx::tc_fence_after();
                    values(1, 1, v, t == 0);
                    commit(&sh.o_full[1]);
                    release(&sh.kv_empty[v]);
                    if (more) {
                        scores(1, 1, k);
                        commit(&sh.s_full[1]);
                        release(&sh.kv_empty[k]);
                        if (t + 2 == n) release(&sh.q_empty);
                    }
                } else {
                    const int now = t & 1;
                    if (more) {
                        if (!arrived(items + 2)) return false;
                        ptx::tc_fence_after();
                        scores(0, now ^ 1, k);
                        commit(&sh.s_full[now ? 0 : 2]);
                        release(&sh.kv_empty[k]);
                        if (t + 2 == n) release(&sh.q_empty);
                    }
                    const uint32_t parity = (now ? p_count[2]++ : p_count[0]++) & 1;
                    if (!arrived(items + 1) || !wait(p, sh, &sh.p_full[now ? 2 : 0], parity)) return false;
                    ptx::tc_fence_after();
                    values(0, now, v, t == 0);
                    commit(&sh.o_full[0]);
                    release(&sh.kv_empty[v]);
                }
            }
        }
    }
};

// ------------------------------------------------------------------------------------------------
// Softmax of one tile of rows, and its output.
template <typename T, int DP, bool kPolled> struct Softmax {
    typedef Sizes<DP> Z;
    typedef Half<T> H;
    static constexpr int kN = Z::kSlots;
    const ChunkParams &p;
    Shared<kPolled> &sh;
    uint32_t tmem;           // of this warp's lanes
    int tile;                // of rows: 0 or 1

    // What this warp has stored to TMEM is there.
    __device__ __forceinline__ void pass_on(uint64_t *bar) {
        ptx::tc_fence_before();
        __syncwarp();
        if (threadIdx.x % 32 == 0) ptx::mbar_arrive(bar);
        __syncwarp();
    }
    // Multiplies this warp's rows of O.
    __device__ __forceinline__ void rescale(float factor) {
        const uint32_t o = tmem + Z::kO + tile * Z::kOPitch;
        for (int d = 0; d < p.D; d += 16) {
            uint32_t v[16];
            tmem_ld16(o + d, v);
            tmem_wait_ld16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * factor);
            tmem_st16(o + d, v);
        }
    }

    __device__ __forceinline__ bool run() {
        const int r = tile * 128 + threadIdx.x % 128;
        // Scores of a negative or zero scale are multiplied before they are compared.
        const bool early = p.scale_log2 <= 0.0f;
        const float scale = early ? 1.0f : p.scale_log2;
        int tiles = 0, o_count = 0, s_count[2] = {0, 0};    // s_count: own barrier, and [2]
        bool ok;
        if (threadIdx.x == 0 && !p.whole) p.heads[blockIdx.x] = make_int4(0, 0, 0, 0);
        for (int no = 0;; ++no) {
            const Segment *const next = next_segment(p, sh, no, ok);
            if (!next) return ok;
            const Segment &u = *next;
            const int n = u.t1 - u.t0, from = (u.first + u.t0) * kN;
            const bool dual = u.rows > 128;
            if (tile == 1 && !dual) {
                tiles += n;
                segment_done(sh, no);
                continue;
            }
            const bool mine = r < u.rows;
            const int hi = mine ? end_slot(p, u.s, (u.r0 + r) / p.G) : 0, lo = first_slot(p, hi);
            float base = kNegInf, l = 0.0f;
            for (int t = 0; t < n; ++t, ++tiles) {
                const bool second = !dual && (t & 1);
                const int buffer = dual ? tile : t & 1, bar = second ? 2 : tile;
                const int j0 = from + t * kN;
                const uint32_t parity = (second ? s_count[1]++ : s_count[0]++) & 1;
                if (!wait(p, sh, &sh.s_full[bar], parity)) return false;
                ptx::tc_fence_after();
                const uint32_t at = tmem + Z::kS + buffer * kN;
                uint32_t seen[kN / 32], all = ~0u;
#pragma unroll
                for (int w = 0; w < kN / 32; ++w) {
                    seen[w] = *(volatile uint32_t *)&sh.visible[tiles % kRing][w];
                    all &= seen[w];
                }
                const bool masked = is_edge(u, j0, kN) || all != ~0u;
                // Scores of 32 slots as the base compares them.
                const auto prepare = [&](uint32_t (&s)[32], int w) {
                    if (early) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s[i] = __float_as_uint(__uint_as_float(s[i]) * p.scale_log2);
                    }
                    if (masked) {
                        const uint32_t bits = seen[w] & range_bits(j0 + w * 32, lo, hi);
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1 ? s[i] : 0xff800000u;
                    }
                };
                float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
                const auto raise_top = [&](const uint32_t (&s)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        top[i / 2 % 4] = max3(top[i / 2 % 4], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                };
                uint32_t s[kN / 32][32];
#pragma unroll
                for (int w = 0; w < kN / 32; ++w) ptx::tmem_ld_32x32b_x32(at + w * 32, s[w]);
#pragma unroll
                for (int w = 0; w < kN / 32; ++w) {
                    ptx::tmem_wait_ld_regs(s[w]);
                    prepare(s[w], w);
                    raise_top(s[w]);
                }
                // Rounded upwards: no power of two below exceeds what the base allows it.
                const float m = __fmul_ru(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), scale);
                const bool raise = m > base + H::kSlack;
                const bool again = raise && base > kNegInf;
                const float factor = again ? shrink_of(base, m) : 1.0f;
                if (raise) base = m;
                // (Before the first of this tile's weights is passed on.)
                if (t > 0 && __any_sync(0xffffffffu, again)) {
                    if (!wait(p, sh, &sh.o_full[tile], (o_count + t - 1) & 1)) return false;
                    ptx::tc_fence_after();
                    rescale(factor);
                }
                const float sub = base == kNegInf ? 0.0f : __fsub_ru(base, H::kLift);
                const uint64_t scale2 = pair(scale, scale), sub2 = pair(-sub, -sub);
                uint64_t sum[2] = {0, 0};
                const auto weigh = [&](const uint32_t (&s)[32], int w) {
                    uint32_t out[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, sub2),
                               a, b);
                        a = pow2(a);
                        b = pow2(b);
                        sum[i % 2] = add2(sum[i % 2], pair(a, b));
                        out[i] = H::pack(a, b);
                    }
                    if (!masked) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) out[i] = H::hold_up(out[i]);
                    }
                    tmem_st16(at + w * 16, out);
                };
#pragma unroll
                for (int w = 0; w < kN / 32; ++w) weigh(s[w], w);
                float even, odd;
                unpair(add2(sum[0], sum[1]), even, odd);
                l = l * factor + (even + odd);
                ptx::tmem_wait_st();
                // The product before the last has to be over before the last can be: the wait behind the
                // loop would take the one's end for the other's.
                if (t == n - 1 && t > 0 && !wait(p, sh, &sh.o_full[tile], (o_count + t - 1) & 1)) return false;
                pass_on(&sh.p_full[bar]);
            }
            o_count += n;
            if (!wait(p, sh, &sh.o_full[tile], (o_count - 1) & 1)) return false;
            ptx::tc_fence_after();
            output(u, r, mine, lo, hi, base, l);
            if (threadIdx.x == 0 && u.part && u.begins)
                p.heads[blockIdx.x] = make_int4(u.b, u.hk, u.m, u.parts);
            segment_done(sh, no);
        }
    }

    __device__ __forceinline__ void output(const Segment &u, int r, bool mine, int lo, int hi, float base,
                                           float l) {
        const bool part = u.part, tainted = *(const volatile int *)&u.taint;
        const uint32_t o = tmem + Z::kO + tile * Z::kOPitch;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (u.begins ? 1 : 0);    // as in Walk
        T *to = (T *)p.out + (mine ? output_offset(p, u, r) : 0);
        if (part && mine) p.part_ml[slot * Z::kRows + r] = make_float2(base, l);
        for (int d = 0; d < p.D; d += 16) {
            uint32_t v[16];
            __syncwarp();
            tmem_ld16(o + d, v);
            tmem_wait_ld16(v);
            if (!mine) continue;
            if (tainted)
                for (int i = 0; i < 16; ++i)
                    v[i] = __float_as_uint(__uint_as_float(v[i]) +
                                           taint_of<T, kN>(p, u, u.t0, u.t1, lo, hi, d + i));
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    p.part_o[(slot * p.D + d + i) * Z::kRows + r] = __uint_as_float(v[i]);
            } else {
                float x[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = l == 0.0f ? 0.0f : __uint_as_float(v[h * 8 + i]) * inv;
                    store8(to + d + h * 8, x);
                }
            }
        }
        __syncwarp();
        // (O has been read when this warp arrives at p_full next.)
    }
};

template <typename T, int DP, bool kPolled> __global__ void __launch_bounds__(kThreads, 1) tc_kernel(ChunkParams p) {
    typedef Sizes<DP> Z;
    extern __shared__ unsigned char dynamic[];
    __shared__ Shared<kPolled> sh;
    const uint32_t raw = ptx::smem_u32(dynamic), smem = (raw + 1023) & ~1023u;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kStages; ++i) {
            ptx::mbar_init(&sh.kv_full[i], 128);
            ptx::mbar_init(&sh.kv_empty[i], 1);
        }
        ptx::mbar_init(&sh.q_full, 128);
        ptx::mbar_init(&sh.q_empty, 1);
        ptx::mbar_init(&sh.drained, 1);
        ptx::mbar_init(&sh.copied, 128);
        for (int i = 0; i < kSegments; ++i) {
            ptx::mbar_init(&sh.segment_full[i], 1);
            ptx::mbar_init(&sh.segment_empty[i], 4 * Z::kTiles + 5);     // warps
        }
        for (int i = 0; i < 3; ++i) {
            ptx::mbar_init(&sh.s_full[i], 2);
            ptx::mbar_init(&sh.p_full[i], 4);
        }
        ptx::mbar_init(&sh.o_full[0], 2);
        ptx::mbar_init(&sh.o_full[1], 2);
        ptx::fence_mbar_init();
        sh.abort = 0;
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&sh.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int64_t *const costs = reinterpret_cast<int64_t *>(dynamic + (smem - raw));    // where Q will be
    sum_costs<Z::kRows, Z::kSlots>(p, costs);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem, q_smem = smem, kv_smem = smem + Z::kQ;
    bool ok = true;
    if (warp < kCopyWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        if (warp / 4 < Z::kTiles) {
            Softmax<T, DP, kPolled> softmax{p, sh, tmem + ((uint32_t)(warp % 4 * 32) << 16), warp / 4};
            ok = softmax.run();
        }
    } else {
        if (warp < kMmaWarp) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
            Copier<T, DP, kPolled> copier{p, sh, q_smem, kv_smem};
            ok = copier.run();
            // Copies that nobody waits for any more: all that this thread began, and their arrivals.
            copier.arrive(&sh.copied);
            ok &= ptx::mbar_wait_warp(&sh.copied, 0, kChunkWaitLimitNs, nullptr);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
            if (warp == kMmaWarp) {
                Multiplier<T, DP, kPolled> multiplier{p, sh, q_smem, kv_smem, tmem};
                ok = multiplier.run();
            } else if (warp == kScheduleWarp) {
                ok = schedule<Z::kRows, Z::kSlots>(p, sh, costs);
            }
        }
    }
    if (!ok) give_up(sh, p);
    if (warp == kMmaWarp) {
        // Products that nobody waits for any more.
        if (ptx::elect_one()) ptx::mma_commit(&sh.drained);
        if (!ptx::mbar_wait_warp(&sh.drained, 0, kChunkWaitLimitNs, nullptr)) give_up(sh, p);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

template <typename T, int DP, bool kPolled>
cudaError_t launch_tc(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    typedef Sizes<DP> Z;
    static_assert(Z::kSmem + sizeof(Shared<kPolled>) <= 227 * 1024, "shared memory");
    static_assert(kMaxB * sizeof(int64_t) <= Z::kQ, "costs");
    static PerDeviceOnce once;
    const auto kernel = tc_kernel<T, DP, kPolled>;
    cudaError_t e = once.run(current_device(), cudaSuccess, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kSmem);
    });
    if (e != cudaSuccess) return e;
    count_launches(1);
    e = launch_pdl(kernel, dim3((unsigned)pl->num_sms), dim3(kThreads), Z::kSmem, st, p);
    if (e != cudaSuccess || p.whole) return e;
    return launch_join<T, Z::kRows>(p, pl->num_sms, st);
}

template <typename T, bool kPolled>
cudaError_t launch_by_size(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    return p.D <= 64 ? launch_tc<T, 64, kPolled>(pl, p, st) : p.D <= 128 ? launch_tc<T, 128, kPolled>(pl, p, st)
                                                                         : launch_tc<T, 256, kPolled>(pl, p, st);
}
template <typename T> cudaError_t launch_16(const ctr_attn_s *pl, const ChunkParams &p, cudaStream_t st) {
    return p.wait_limit_ns == kChunkWaitLimitNs ? launch_by_size<T, false>(pl, p, st)
                                                : launch_by_size<T, true>(pl, p, st);
}

}  // namespace chunk
}  // namespace ctr
