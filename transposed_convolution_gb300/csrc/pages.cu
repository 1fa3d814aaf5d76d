// pages.cu -- pages of the cache for new tokens, and their slots and positions (ctr_pages_*).
//
// A reservation is two prefix sums over at most 1024 sequences (pages needed, tokens granted) and
// then independent stores: 12 bytes a token and 4 a page, against a free list that is only read.
// Its time is the launch and the chain of loads and scans, not its bytes, so it is one launch:
// every block sums up all sequences by itself (8 KB from L2) instead of waiting for another,
// and writes its share of the rows and pages; pages that the call itself takes are read from the
// list, never from the table, so no block reads what another one writes.  Only the free list's
// count changes under the blocks' eyes: the last one to finish writes it.
// In a captured graph, given back and reserved: 64 sequences of one token 8.7 us, 256 of 1000 16.5.
#include <algorithm>
#include <cstdio>
#include <new>

#include "decode_internal.h"
#include "ptx.cuh"

struct ctr_pages_s {
    int64_t B, page, max_pages;
    int32_t *free_pages, *count;
    int64_t num_pages;
    void *ws;
    int ready;
};

namespace ctr {
namespace {

constexpr int kThreads = 256, kMaxB = 1024, kPer = kMaxB / kThreads;
constexpr int kRowsABlock = 1024;

struct PagesParams {
    int32_t *tables;
    const int32_t *lens, *counts;       // counts: tokens to add, or tokens to keep
    int32_t *granted, *starts, *positions, *lens_out;
    int64_t *slots;
    int64_t rows;
    int32_t *free_pages, *count;
    uint32_t *status, *ticket;
    int B, page, max_pages, num_pages, cap;
};

struct Two {
    int64_t pages, tokens;
};

// The exclusive prefix sums of v over the block's threads, and the totals.  Every thread calls it.
__device__ __noinline__ Two block_scan(Two v, Two *total) {
    __shared__ Two sums[kThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Two up = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, up.pages, d);
        const int64_t y = __shfl_up_sync(0xffffffffu, up.tokens, d);
        if (lane >= d) {
            up.pages += x;
            up.tokens += y;
        }
    }
    __syncthreads();                    // the sums of an earlier call have been read
    if (lane == 31) sums[warp] = up;
    __syncthreads();
    Two before = {0, 0}, all = {0, 0};
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = all;
        all.pages += sums[w].pages;
        all.tokens += sums[w].tokens;
    }
    *total = all;
    return {before.pages + up.pages - v.pages, before.tokens + up.tokens - v.tokens};
}

// The last i with from[i] <= x, of n ascending numbers with from[0] <= x.
__device__ __forceinline__ int find(const int64_t *from, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (from[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page) {
    return tokens / page + (tokens % page != 0);
}

// Pages on the free list.  A count out of range is reported and cut.
__device__ __forceinline__ int free_count(const PagesParams &p) {
    const int c = *p.count;
    if ((unsigned)c <= (unsigned)p.num_pages) return c;
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadLength);
    return c < 0 ? 0 : p.num_pages;
}

// The last block to finish writes the list's new count.
__device__ __forceinline__ void finish(const PagesParams &p, int count) {
    __syncthreads();                    // this block has read the old count
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(p.ticket, 1u) == gridDim.x - 1) {
            __threadfence();
            *p.count = count;
            *p.ticket = 0;
        }
    }
}

__global__ void __launch_bounds__(kThreads) reserve_kernel(PagesParams p) {
    // Of each sequence: its first row, its first page's place among those taken, its length.
    __shared__ int64_t starts[kMaxB + 1], taken[kMaxB + 1];
    __shared__ int lens[kMaxB];
    const int t = threadIdx.x;
    ptx::griddep_wait();
    const int have = free_count(p);
    int len[kPer], n[kPer], need[kPer];
    Two sum = {0, 0}, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = t * kPer + i;
        len[i] = b < p.B ? p.lens[b] : -1;
        n[i] = b < p.B && len[i] >= 0 ? p.counts[b] : 0;
        if (n[i] < 0 || len[i] > p.cap || n[i] > p.cap - len[i]) {
            if (blockIdx.x == 0) atomicOr(p.status, kStatusBadLength);
            n[i] = 0;
        }
        need[i] = n[i] ? pages_of(len[i] + n[i], p.page) - pages_of(len[i], p.page) : 0;
        sum.pages += need[i];
        sum.tokens += n[i];
    }
    // First come, first served: a request is granted if the pages (unless it needs none) and the
    // rows of all requests up to it are there.
    Two at = block_scan(sum, &total);
    sum = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        at.pages += need[i];
        at.tokens += n[i];
        if ((need[i] && at.pages > have) || at.tokens > p.rows) n[i] = need[i] = 0;
        sum.pages += need[i];
        sum.tokens += n[i];
    }
    at = block_scan(sum, &total);
    const int64_t pages = total.pages, granted_rows = total.tokens;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = t * kPer + i;
        if (b < p.B) {
            starts[b] = at.tokens;
            taken[b] = at.pages;
            lens[b] = len[i];
            if (blockIdx.x == 0) {
                p.granted[b] = n[i];
                p.starts[b] = (int)at.tokens;
                p.lens_out[b] = len[i] + n[i];
            }
        }
        at.tokens += n[i];
        at.pages += need[i];
    }
    if (t == 0) {
        starts[p.B] = granted_rows;
        taken[p.B] = pages;
        if (blockIdx.x == 0) p.starts[p.B] = (int)granted_rows;
    }
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + t;
    for (int64_t i = me; i < p.rows; i += step) {
        int64_t slot = -1;
        int pos = 0;
        if (i < granted_rows) {
            const int b = find(starts, p.B, i);
            pos = lens[b] + (int)(i - starts[b]);
            const int pg = pos / p.page, own = pg - pages_of(lens[b], p.page);
            const int no = own < 0 ? p.tables[(int64_t)b * p.max_pages + pg]
                                   : p.free_pages[have - 1 - (taken[b] + own)];
            if ((unsigned)no < (unsigned)p.num_pages)
                slot = (int64_t)no * p.page + pos % p.page;
            else
                atomicOr(p.status, kStatusBadPage);
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
    for (int64_t i = me; i < pages; i += step) {
        const int b = find(taken, p.B, i);
        int no = p.free_pages[have - 1 - i];
        if ((unsigned)no >= (unsigned)p.num_pages) {
            atomicOr(p.status, kStatusBadPage);
            no = -1;
        }
        p.tables[(int64_t)b * p.max_pages + pages_of(lens[b], p.page) + (i - taken[b])] = no;
    }
    finish(p, have - (int)pages);
}

// The tail pages of every sequence back to the list, the last sequence's last page first: what is given
// back comes out again in the order it had.
__global__ void __launch_bounds__(kThreads) release_kernel(PagesParams p) {
    __shared__ int64_t given[kMaxB + 1];
    __shared__ int first[kMaxB];
    const int t = threadIdx.x;
    ptx::griddep_wait();
    const int have = free_count(p);
    int pages[kPer];
    Two mine = {0, 0}, sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = t * kPer + i;
        pages[i] = 0;
        if (b >= p.B) continue;
        int len = p.lens[b];
        const int keep = p.counts[b];
        int left = len;
        if (len > p.cap) {
            if (blockIdx.x == 0) atomicOr(p.status, kStatusBadLength);
            len = p.cap;
        }
        if (len >= 0 && keep < len) {
            left = keep < 0 ? -1 : keep;
            first[b] = pages_of(max(keep, 0), p.page);
            pages[i] = pages_of(len, p.page) - first[b];
        }
        if (blockIdx.x == 0) p.lens_out[b] = left;
        mine.pages += pages[i];
    }
    int64_t at = block_scan(mine, &sum).pages;
    const int64_t total = sum.pages;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (t * kPer + i < p.B) given[t * kPer + i] = at;
        at += pages[i];
    }
    if (t == 0) given[p.B] = total;
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + t; i < total; i += step) {
        const int b = find(given, p.B, i);
        int32_t *entry = p.tables + (int64_t)b * p.max_pages + first[b] + (i - given[b]);
        const int no = *entry;
        const int64_t to = have + total - 1 - i;
        if ((unsigned)no >= (unsigned)p.num_pages) atomicOr(p.status, kStatusBadPage);
        *entry = -1;
        if (to < p.num_pages) p.free_pages[to] = no;
        else atomicOr(p.status, kStatusBadLength);   // more pages than there are: some given back twice
    }
    finish(p, (int)min(have + total, (int64_t)p.num_pages));
}

__global__ void __launch_bounds__(kThreads) fill_kernel(PagesParams p) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    ptx::griddep_wait();
    if (i < p.num_pages) p.free_pages[i] = p.num_pages - 1 - (int)i;
    if (i == 0) *p.count = p.num_pages;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

ctr_status ready(const ctr_pages_s *pl) {
    if (!pl->free_pages) return CTR_ERR_NOT_PREPARED;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    return pl->ready ? CTR_OK : CTR_ERR_NOT_PREPARED;
}

PagesParams params_of(const ctr_pages_s *pl) {
    PagesParams p = {};
    p.free_pages = pl->free_pages;
    p.count = pl->count;
    p.status = static_cast<uint32_t *>(pl->ws);
    p.ticket = p.status + 32;
    p.B = (int)pl->B;
    p.page = (int)pl->page;
    p.max_pages = (int)pl->max_pages;
    p.num_pages = (int)pl->num_pages;
    p.cap = (int)(pl->page * pl->max_pages);
    return p;
}

}  // namespace
}  // namespace ctr

extern "C" {

ctr_status ctr_pages_create(ctr_pages_t *out, int64_t B, int64_t page_size, int64_t max_pages) {
    if (!out) return CTR_ERR_INVALID_ARG;
    *out = nullptr;
    if (B < 1 || page_size < 1 || max_pages < 1) return CTR_ERR_INVALID_ARG;
    const int64_t cap = (int64_t)1 << 28;
    if (B > ctr::kMaxB || page_size > cap || max_pages > cap / page_size) return CTR_ERR_UNSUPPORTED;
    ctr_pages_s *pl = new (std::nothrow) ctr_pages_s();
    if (!pl) return CTR_ERR_INVALID_ARG;
    pl->B = B;
    pl->page = page_size;
    pl->max_pages = max_pages;
    *out = pl;
    return CTR_OK;
}

ctr_status ctr_pages_bind_list(ctr_pages_t pl, int32_t *free_pages, int32_t *count, int64_t num_pages) {
    if (!pl || !free_pages || !count || free_pages == count || num_pages < 1) return CTR_ERR_INVALID_ARG;
    if (num_pages > 0x7fffffff) return CTR_ERR_UNSUPPORTED;
    if (!ctr::aligned(free_pages, 4) || !ctr::aligned(count, 4)) return CTR_ERR_MISALIGNED;
    pl->free_pages = free_pages;
    pl->count = count;
    pl->num_pages = num_pages;
    return CTR_OK;
}

size_t ctr_pages_workspace_bytes(ctr_pages_t pl) { return pl ? 256 : 0; }

ctr_status ctr_pages_bind_workspace(ctr_pages_t pl, void *ws, size_t bytes) {
    if (!pl || !ws) return CTR_ERR_INVALID_ARG;
    if (!ctr::aligned(ws, 256)) return CTR_ERR_MISALIGNED;
    if (bytes < 256) return CTR_ERR_NO_WORKSPACE;
    pl->ws = ws;
    pl->ready = 0;
    return CTR_OK;
}

ctr_status ctr_pages_reset(ctr_pages_t pl, int refill, void *stream) {
    if (!pl || (refill != 0 && refill != 1)) return CTR_ERR_INVALID_ARG;
    if (!pl->free_pages) return CTR_ERR_NOT_PREPARED;
    if (!pl->ws) return CTR_ERR_NO_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(pl->ws, 0, 256, st) != cudaSuccess) return CTR_ERR_CUDA;
    if (refill) {
        const ctr::PagesParams p = ctr::params_of(pl);
        const int64_t blocks = (pl->num_pages + ctr::kThreads - 1) / ctr::kThreads;
        ctr::count_launches(1);
        if (ctr::launch_pdl(ctr::fill_kernel, dim3((unsigned)blocks), dim3(ctr::kThreads), 0, st, p) !=
            cudaSuccess)
            return CTR_ERR_CUDA;
    }
    pl->ready = 1;
    return CTR_OK;
}

ctr_status ctr_pages_reserve(ctr_pages_t pl, int32_t *tables, const int32_t *lens, const int32_t *counts,
                             int64_t rows, int32_t *granted, int32_t *starts, int64_t *slots,
                             int32_t *positions, int32_t *lens_out, void *stream) {
    if (!pl || !tables || !lens || !counts || rows < 0 || !granted || !starts || !lens_out ||
        (rows && (!slots || !positions)))
        return CTR_ERR_INVALID_ARG;
    if (lens_out == lens || lens_out == counts || granted == lens || granted == counts || granted == lens_out)
        return CTR_ERR_INVALID_ARG;
    if (rows > ((int64_t)1 << 30)) return CTR_ERR_UNSUPPORTED;
    for (const void *a : {(const void *)tables, (const void *)lens, (const void *)counts, (const void *)granted,
                          (const void *)starts, (const void *)positions, (const void *)lens_out})
        if (!ctr::aligned(a, 4)) return CTR_ERR_MISALIGNED;
    if (!ctr::aligned(slots, 8)) return CTR_ERR_MISALIGNED;
    if (const ctr_status s = ctr::ready(pl)) return s;
    ctr::PagesParams p = ctr::params_of(pl);
    p.tables = tables;
    p.lens = lens;
    p.counts = counts;
    p.granted = granted;
    p.starts = starts;
    p.slots = slots;
    p.positions = positions;
    p.lens_out = lens_out;
    p.rows = rows;
    // A block for each 1024 rows (the scan costs as much as storing that many), two an SM at most.
    const int64_t blocks = std::min<int64_t>(2 * ctr::device_sms(),
                                             1 + rows / ctr::kRowsABlock);
    ctr::count_launches(1);
    return ctr::launch_pdl(ctr::reserve_kernel, dim3((unsigned)blocks), dim3(ctr::kThreads), 0,
                           static_cast<cudaStream_t>(stream), p) == cudaSuccess ? CTR_OK : CTR_ERR_CUDA;
}

ctr_status ctr_pages_release(ctr_pages_t pl, int32_t *tables, const int32_t *lens, const int32_t *keep,
                             int32_t *lens_out, void *stream) {
    if (!pl || !tables || !lens || !keep || !lens_out || lens_out == lens || lens_out == keep)
        return CTR_ERR_INVALID_ARG;
    for (const void *a : {(const void *)tables, (const void *)lens, (const void *)keep, (const void *)lens_out})
        if (!ctr::aligned(a, 4)) return CTR_ERR_MISALIGNED;
    if (const ctr_status s = ctr::ready(pl)) return s;
    ctr::PagesParams p = ctr::params_of(pl);
    p.tables = tables;
    p.lens = lens;
    p.counts = keep;
    p.lens_out = lens_out;
    // How many pages come back is on the device; at most what the list holds.
    const int64_t most = std::min(pl->num_pages, pl->B * pl->max_pages);
    const int64_t blocks = std::min<int64_t>(2 * ctr::device_sms(), 1 + most / (8 * ctr::kRowsABlock));
    ctr::count_launches(1);
    return ctr::launch_pdl(ctr::release_kernel, dim3((unsigned)blocks), dim3(ctr::kThreads), 0,
                           static_cast<cudaStream_t>(stream), p) == cudaSuccess ? CTR_OK : CTR_ERR_CUDA;
}

ctr_status ctr_pages_check(ctr_pages_t pl, void *stream) {
    if (!pl) return CTR_ERR_INVALID_ARG;
    if (const ctr_status s = ctr::ready(pl)) return s;
    return ctr::check_status(pl->ws, static_cast<cudaStream_t>(stream));
}

ctr_status ctr_pages_describe(ctr_pages_t pl, char *buf, size_t len) {
    if (!pl || !buf || len == 0) return CTR_ERR_INVALID_ARG;
    snprintf(buf, len, "pages B=%lld page=%lld max_pages=%lld num_pages=%lld", (long long)pl->B,
             (long long)pl->page, (long long)pl->max_pages, (long long)pl->num_pages);
    return CTR_OK;
}

void ctr_pages_destroy(ctr_pages_t pl) { delete pl; }

}  // extern "C"
