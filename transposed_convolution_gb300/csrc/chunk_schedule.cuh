// chunk_schedule.cuh -- which rows and slots a block of the chunk attention takes.
//
// A unit is one sequence, KV head and tile of MT query rows, row r of a sequence being token r / G
// and head r % G of the KV head's group, so that the heads that share K and V share its tiles.  A
// unit's slots come in tiles of NT.  All units' tiles, in a row, are cut into equal chunks, one for
// each block (entering a unit counts as one tile more), so ragged batches, long prompts and a
// few tokens on a long cache fill the GPU alike.  The parts of a unit that several chunks share are
// joined in chunk order by a second kernel, so results do not depend on timing.
// Lengths are on the device, so every block finds its place by itself: a sum over all units first
// (a lane a unit, a few instructions), then a search.
#pragma once

#include "decode_device.cuh"
#include "ptx.cuh"

namespace ctr {
namespace chunk {

constexpr int kMaxB = 1024;

// One sequence's share of the call.
struct Sequence {
    int row0, n, len;        // first row of q, new tokens, tokens before them (< 0: idle)
};

// Reports starts or lengths out of range, from the first block.
__device__ __forceinline__ Sequence sequence_of(const ChunkParams &p, int b, bool report) {
    Sequence s;
    const int s0 = p.starts[b], s1 = p.starts[b + 1];
    s.row0 = s0;
    s.n = s1 - s0;
    s.len = p.cache.lens[b];
    if (s0 < 0 || s1 < s0 || s1 > p.T) {
        if (report && blockIdx.x == 0) atomicOr(p.cache.status, kStatusBadLength);
        s.row0 = s.n = 0;
    }
    // (An idle sequence asks for no slots, whatever its rows.)
    if (s.len >= 0 && s.len > p.cache.cap - s.n) {
        if (report && blockIdx.x == 0) atomicOr(p.cache.status, kStatusBadLength);
        s.len = min(s.len, p.cache.cap);
    }
    return s;
}

// Token t of a sequence attends to the slots [first, end).
__device__ __forceinline__ int end_slot(const ChunkParams &p, const Sequence &s, int t) {
    return s.len < 0 ? 0 : min(s.len + t + 1, p.cache.cap);
}
__device__ __forceinline__ int first_slot(const ChunkParams &p, int end) {
    return p.window > 0 && end > p.window ? end - (int)p.window : 0;
}

template <int MT, int NT> struct Unit {
    Sequence s;
    int b, hk, m, units;     // sequence, KV head, tile of rows, tiles of rows of the sequence
    int r0, rows;            // first row in the sequence, rows (up to MT)
    int lo, hi;              // slots that any row attends to
    int lo_last, hi_first;   // slots in [lo_last, hi_first) are attended to by every row
    int first, tiles;        // tiles of slots, one at least

    __device__ __forceinline__ void tile(const ChunkParams &p) {
        r0 = m * MT;
        rows = min(MT, s.n * p.G - r0);
        hi_first = end_slot(p, s, r0 / p.G);
        hi = end_slot(p, s, (r0 + rows - 1) / p.G);
        lo = first_slot(p, hi_first);
        lo_last = first_slot(p, hi);
        first = lo / NT;
        tiles = max(1, (hi + NT - 1) / NT - first);
    }
};

// Tiles and entries of a sequence's units of one KV head; the lanes of a warp share them.
template <int MT, int NT> __device__ __forceinline__ int64_t sequence_cost(const ChunkParams &p, int b) {
    Unit<MT, NT> u;
    u.s = sequence_of(p, b, threadIdx.x % 32 == 0);
    const int units = (int)(((int64_t)u.s.n * p.G + MT - 1) / MT);
    int64_t sum = 0;
    for (u.m = threadIdx.x % 32; u.m < units; u.m += 32) {
        u.tile(p);
        sum += u.tiles + 1;
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// a / b, a >= 0 and b > 0: mostly both have 32 bits, whose division takes a fifth of the time.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Where a block begins.
struct Start {
    int64_t x, x1;           // this block's stretch of all units' tiles and entries
    int64_t unit;            // where the first unit lies
    int64_t chunk;           // length of every block's stretch
    int b, hk, m;
};

// A walk over the units of a block's chunk.
template <int MT, int NT> struct Walk {
    Unit<MT, NT> u;
    int64_t unit, x, x1, chunk;
    // Segment: tiles [t0, t1) of the unit, not all of them if it is a part.
    int t0, t1;
    bool part, begins;       // begins: the unit's first tile is in it

    __device__ __forceinline__ void start(const ChunkParams &p, const Start &s) {
        x = s.x;
        x1 = s.x1;
        unit = s.unit;
        chunk = s.chunk;
        u.b = s.b;
        u.hk = s.hk;
        u.m = s.m;
        if (x < x1) enter(p);
    }
    __device__ __forceinline__ void enter(const ChunkParams &p) {
        u.s = sequence_of(p, u.b, false);
        u.units = (int)(((int64_t)u.s.n * p.G + MT - 1) / MT);
        u.tile(p);
    }
    // The next segment, if there is one.
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        while (x < x1) {
            const int64_t tiles = unit + 1, end = tiles + u.tiles;
            if (x >= end) {
                unit = end;
                if (!advance(p)) break;
                continue;
            }
            if (p.whole) {       // units that begin in the stretch, and all of them
                const bool ours = x == unit;
                t0 = 0;
                t1 = u.tiles;
                part = false;
                begins = true;
                x = end;
                if (ours) return true;
                continue;
            }
            t0 = (int)(max(x, tiles) - tiles);
            t1 = (int)(min(x1, end) - tiles);
            part = t0 > 0 || t1 < u.tiles;
            begins = t0 == 0;
            x = min(x1, end);
            if (t1 > t0) return true;
        }
        return false;
    }
    // On to the next unit.
    __device__ __forceinline__ bool advance(const ChunkParams &p) {
        if (++u.m < u.units) {
            u.tile(p);
            return true;
        }
        u.m = 0;
        if (++u.hk < p.Hkv) {
            u.tile(p);
            return true;
        }
        u.hk = 0;
        do {
            if (++u.b >= p.B) return false;
            u.s = sequence_of(p, u.b, false);
        } while (u.s.n == 0);
        enter(p);
        return true;
    }
    // Where a part goes: a block has one at most that begins before its stretch, and one that does not.
    __device__ __forceinline__ int64_t slot() const { return 2 * (int64_t)blockIdx.x + (begins ? 1 : 0); }
    // Parts of the unit whose first one this is.
    __device__ __forceinline__ int parts() const {
        return (int)divide(unit + u.tiles, chunk) - (int)blockIdx.x + 1;
    }
};

// The sequences' costs (of one KV head), by all warps of the block; for a barrier to follow.
template <int MT, int NT> __device__ __forceinline__ void sum_costs(const ChunkParams &p, int64_t *costs) {
    for (int b = threadIdx.x / 32; b < p.B; b += blockDim.x / 32) {
        const int64_t c = sequence_cost<MT, NT>(p, b);
        if (threadIdx.x % 32 == 0) costs[b] = c;
    }
}

// Finds the block's start; one warp calls it.
template <int MT, int NT> __device__ __forceinline__ Start find_start(const ChunkParams &p, const int64_t *costs) {
    const int lane = threadIdx.x % 32;
    int64_t all = 0;
    for (int b = lane; b < p.B; b += 32) all += costs[b];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) all += __shfl_xor_sync(0xffffffffu, all, d);
    all *= p.Hkv;
    Start s;
    s.chunk = divide(all + gridDim.x - 1, gridDim.x);
    s.x = min(all, s.chunk * blockIdx.x);
    s.x1 = min(all, s.x + s.chunk);
    s.unit = s.b = s.hk = s.m = 0;
    if (s.x < s.x1) {
        // The sequence: thirty-two at a time.
        int64_t before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int64_t c = b0 + lane < p.B ? costs[b0 + lane] * p.Hkv : 0;
            int64_t up = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t v = __shfl_up_sync(0xffffffffu, up, d);
                if (lane >= d) up += v;
            }
            const unsigned here = __ballot_sync(0xffffffffu, before + up > s.x);
            const int at = here ? __ffs(here) - 1 : 31;
            const int64_t own = __shfl_sync(0xffffffffu, c, at), upto = __shfl_sync(0xffffffffu, up, at);
            if (here) {
                s.b = b0 + at;
                before += upto - own;
                break;
            }
            before += upto;
        }
        const int64_t cost = costs[s.b];
        s.hk = (int)divide(s.x - before, cost);
        before += s.hk * cost;
        // The tile of rows.
        Unit<MT, NT> u;
        u.s = sequence_of(p, s.b, false);
        u.units = (int)(((int64_t)u.s.n * p.G + MT - 1) / MT);
        for (int m0 = 0; m0 < u.units; m0 += 32) {
            int64_t c = 0;
            u.m = m0 + lane;
            if (u.m < u.units) {
                u.tile(p);
                c = u.tiles + 1;
            }
            int64_t up = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t v = __shfl_up_sync(0xffffffffu, up, d);
                if (lane >= d) up += v;
            }
            const unsigned here = __ballot_sync(0xffffffffu, before + up > s.x);
            const int at = here ? __ffs(here) - 1 : 31;
            const int64_t own = __shfl_sync(0xffffffffu, c, at), upto = __shfl_sync(0xffffffffu, up, at);
            if (here) {
                s.m = m0 + at;
                s.unit = before + upto - own;
                break;
            }
            before += upto;
        }
    }
    return s;
}

}  // namespace chunk
}  // namespace ctr
