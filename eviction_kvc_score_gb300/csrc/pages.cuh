// pages.cuh -- what the calls that move rows of page lists share, whatever a row
// is made of (pages.cu, pages_quant.cu): the plan of a call, the search for the
// list that a row of the flat sequence belongs to, and where a row goes.
#pragma once

#include "cache.cuh"

namespace kvc {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;

struct PlanParams {
    PagesState s;
    int32_t *table, *len;
    const int32_t *counts;
    const int64_t *src_row;   // append only
    int64_t src_step, src_rows;
    int32_t n_lists, n_pages, max_pages, shift, k_max;
    bool append;
};

struct Two {
    int64_t rows, pages;
};

__device__ __forceinline__ Two operator+(Two a, Two b) { return {a.rows + b.rows, a.pages + b.pages}; }

// Exclusive scan over the block; *total receives the sum.  scratch: 33 entries.
__device__ inline Two block_scan(Two v, Two *scratch, Two *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Two x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Two y{__shfl_up_sync(0xffffffffu, x.rows, d), __shfl_up_sync(0xffffffffu, x.pages, d)};
        if (lane >= d) x = x + y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        Two w = lane < (int)(blockDim.x >> 5) ? scratch[lane] : Two{0, 0};
        const Two own = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Two y{__shfl_up_sync(0xffffffffu, w.rows, d), __shfl_up_sync(0xffffffffu, w.pages, d)};
            if (lane >= d) w = w + y;
        }
        if (lane == 31) scratch[32] = w;
        scratch[lane] = {w.rows - own.rows, w.pages - own.pages};
    }
    __syncthreads();
    const Two r{scratch[warp].rows + x.rows - v.rows, scratch[warp].pages + x.pages - v.pages};
    *total = scratch[32];
    __syncthreads();
    return r;
}

// Where rows come from and go to: the running call's plan, and its lists.
struct MoveLists {
    PagesState s;
    int32_t *table;
    const int64_t *src_row;   // append: rows of the source
    int64_t src_step;
    const int32_t *idx;       // compact: rows of the list itself
    int32_t n_lists, n_pages, max_pages, shift, k_max;
};

// Last i of [0, n) with begin[i] <= x (begin ascends from 0); the whole warp
// asks for one x, 32 places at a time.
template <typename T>
__device__ __forceinline__ int owner(const T *begin, int n, T x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, span = n;
    while (span > 1) {
        const int step = (span + 31) >> 5, i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, lane * step < span && begin[i] <= x);
        const int k = 31 - __clz(below);
        span = min(step, span - k * step);
        lo += k * step;
    }
    return lo;
}

// The same for one lane that knows an i with begin[i] <= x: the next list's where x
// is past it, further on by doubled steps and halving, because lists without rows
// (all but one sequence's, when that sequence's prompt is appended) may stand
// between by the hundred thousand (2 x 12,000 rows in 262,144 lists: 15.5 ms one
// list after the other, 0.43 so).
template <typename T>
__device__ __forceinline__ int owner_from(const T *begin, int n, T x, int i) {
    if (i + 1 >= n || begin[i + 1] > x) return i;
    int lo = i + 1, step = 1;
    while (lo + step < n && begin[lo + step] <= x) {
        lo += step;
        step = min(2 * step, n);
    }
    for (int hi = min(n, lo + step); hi - lo > 1;) {
        const int mid = lo + (hi - lo) / 2;
        if (begin[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The new pages' table entries of an append, 32 a warp; warp `me` of `warps`.
__device__ __forceinline__ void enter_pages(const MoveLists &p, int64_t me, int64_t warps) {
    const int lane = threadIdx.x & 31, ps = 1 << p.shift;
    const int total_new = p.s.head->total_new;
    for (int64_t e0 = me * 32; e0 < total_new; e0 += warps * 32) {
        int i = owner(p.s.page_begin, p.n_lists, (int32_t)e0);
        const int e = (int)e0 + lane;
        if (e >= total_new) continue;
        i = owner_from(p.s.page_begin, p.n_lists, (int32_t)e, i);
        const int32_t len = p.s.old_len[i];
        const int first = p.s.shared[i] >= 0 ? len >> p.shift : (len + ps - 1) >> p.shift;
        p.table[(int64_t)i * p.max_pages + first + (e - p.s.page_begin[i])] = p.s.fresh[e];
    }
    __syncwarp();
}

struct MovedRow {
    int64_t from, to;   // from: -1 for a row of zeros
    bool own_pool;      // from counts the pool's rows, not the source's
};

// Row r of the flat sequence, which is list i's.
template <bool APPEND>
__device__ __forceinline__ MovedRow moved_row(const MoveLists &p, int i, int64_t r, uint32_t *bad) {
    const int ps = 1 << p.shift;
    const int64_t *begin = p.s.row_begin;
    int32_t at = (int32_t)(r - begin[i]);   // row within the list's moved rows
    const int32_t *fresh = p.s.fresh + p.s.page_begin[i];
    const int32_t *entry = p.table + (int64_t)i * p.max_pages;
    int64_t from = -1, to;
    bool own_pool = true;
    if (APPEND) {
        const int32_t len = p.s.old_len[i], shared = p.s.shared[i], fill = len & (ps - 1);
        const int first = shared >= 0 ? len >> p.shift : (len + ps - 1) >> p.shift;
        int32_t pos;
        if (shared >= 0 && at < fill) {
            from = ((int64_t)shared << p.shift) + at;
            pos = (len - fill) + at;
        } else {
            if (shared >= 0) at -= fill;
            from = p.src_row[i] + at * p.src_step;
            own_pool = false;
            pos = len + at;
        }
        const int slot = pos >> p.shift;
        const int32_t page = slot >= first ? fresh[slot - first] : entry[slot];
        to = ((int64_t)page << p.shift) + (pos & (ps - 1));
    } else {
        const int32_t src = p.idx[(int64_t)i * p.k_max + at];
        if (src >= 0 && src < p.s.old_len[i]) {
            const int32_t page = entry[src >> p.shift];
            if (page >= 0 && page < p.n_pages)
                from = ((int64_t)page << p.shift) + (src & (ps - 1));
            else
                *bad |= KVC_DEV_BAD_PAGE;
        } else {
            *bad |= KVC_DEV_BAD_LIST;
        }
        to = ((int64_t)fresh[at >> p.shift] << p.shift) + (at & (ps - 1));
    }
    return {from, to, own_pool};
}

inline int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

void launch_pages_plan(const PlanParams &p, cudaStream_t st);
// After a compaction's rows have moved.
void launch_pages_swap(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len, int32_t n_lists,
                       const int32_t *counts, cudaStream_t st);

}  // namespace kvc
