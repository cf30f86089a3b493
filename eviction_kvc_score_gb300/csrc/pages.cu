// pages.cu -- appending to, forking, compacting and cutting the page lists of
// a paged cache.
//
// Taking pages has to give the same pages every time, whatever order blocks
// run in: the free pages of the lowest numbers, in list order.  One block
// plans a call: it counts the pages and rows of every list, scans both counts,
// walks the free bitmap up to as many pages as are needed and writes their
// numbers down; nothing is changed unless all of it fits.  Every SM then moves
// the rows, each warp a run of the flat sequence of all lists' rows, so one
// long list is spread as well as many short ones.  Letting go of pages needs
// no order: holders are counted down by atomics and a page whose count reaches
// zero gets its bit, which commute.
//
// The moves are bound by HBM: 560,000 rows of 128 bf16 (K and V, read and
// written: 573 MB) in 90 us with cold caches, 6.3 TB/s or 93% of the measured copy
// rate.  The plan is a chain of memory latencies, 7 us for a few pages and 12 us
// for 9,000 with cold caches; while each thread wrote down the pages of its own word
// it took 4 us more.
#include "cache.cuh"

namespace kvc {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kListThreads = 128;

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
__device__ Two block_scan(Two v, Two *scratch, Two *total) {
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

// Count a page's holder away; pages nobody holds become free.  Every thread of
// the warp calls it (page < 0: nothing to let go of).
__device__ void let_go(const PagesState &s, int32_t page, int32_t n_pages) {
    const int lane = threadIdx.x & 31;
    bool freed = false;
    if (page >= n_pages) {
        set_status(&s.head->status, KVC_DEV_BAD_PAGE);
    } else if (page >= 0) {
        const int32_t was = atomicSub(&s.holders[page], 1);
        freed = was == 1;
        if (was <= 0) {   // held by nobody: undo
            atomicAdd(&s.holders[page], 1);
            set_status(&s.head->status, KVC_DEV_BAD_PAGE);
        }
        if (freed) atomicOr(&s.bitmap[page >> 5], 1u << (page & 31));
    }
    const int group = freed ? page / kGroupPages : -1;
    const unsigned same = __match_any_sync(0xffffffffu, group);
    if (freed && lane == __ffs(same) - 1) {
        atomicAdd(&s.group_free[group], __popc(same));
        atomicAdd(&s.head->n_free, __popc(same));
    }
}

__global__ void pages_init_kernel(PagesState s, int32_t n_pages) {
    let_next_start();
    wait_for_inputs();
    const int stride = gridDim.x * blockDim.x, me = blockIdx.x * blockDim.x + threadIdx.x;
    for (int w = me; w < s.n_words; w += stride) {
        const int left = n_pages - w * 32;
        s.bitmap[w] = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
    }
    for (int64_t p = me; p < n_pages; p += stride) s.holders[p] = 0;
    for (int g = me; g < s.n_groups; g += stride)
        s.group_free[g] = min(kGroupPages, n_pages - g * kGroupPages);
    if (me == 0) {
        *s.head = PagesHeader{0, n_pages, 0, 0, 0};
    }
}

// What the plan knows of a list.
struct ListPlan {
    int32_t n, len, shared;   // rows to move, length, last page to copy from (or -1)
};

// Pages and rows of list i, and what stands against the call.
__device__ Two list_needs(const PlanParams &p, int i, uint32_t *bad, ListPlan *list) {
    const int32_t n = p.counts[i], len = p.len[i], ps = 1 << p.shift;
    const int64_t row = p.append ? p.src_row[i] : 0;
    const int64_t most = (int64_t)p.max_pages << p.shift;
    Two need{0, 0};
    *list = ListPlan{n, len, -1};
    if (p.append ? n <= 0 : n < 0) return need;
    if (len < 0 || len > most) {
        *bad |= KVC_DEV_BAD_LIST;
        return need;
    }
    need.rows = n;
    if (!p.append) {
        if (n > p.k_max) *bad |= KVC_DEV_BAD_LIST;
        if (n > most) *bad |= KVC_DEV_PAGES_FULL;
        need.pages = (n + ps - 1) >> p.shift;
        return need;
    }
    const int64_t now = (int64_t)len + n;
    if (now > most) {
        *bad |= KVC_DEV_PAGES_FULL;
        return need;
    }
    // (n - 1) * step may pass 64 bits: compare by division
    if (row < 0 || row >= p.src_rows ||
        (n > 1 && p.src_step > 0 && n - 1 > (p.src_rows - 1 - row) / p.src_step)) {
        *bad |= KVC_DEV_BAD_LIST;
        return need;
    }
    need.pages = (int32_t)((now + ps - 1) >> p.shift) - ((len + ps - 1) >> p.shift);
    if (len & (ps - 1)) {
        const int32_t last = p.table[(int64_t)i * p.max_pages + (len >> p.shift)];
        if (last < 0 || last >= p.n_pages) {
            *bad |= KVC_DEV_BAD_PAGE;
        } else if (p.s.holders[last] > 1) {
            list->shared = last;
            need.pages += 1;
            need.rows += len & (ps - 1);
        }
    }
    return need;
}

// The n-th (from 0) set bit of x.
__device__ __forceinline__ int nth_bit(uint32_t x, int n) {
    int at = 0;
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        const int below = __popc((x >> at) & ((1u << w) - 1u));
        if (n >= below) {
            n -= below;
            at += w;
        }
    }
    return at;
}

__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(PlanParams p) {
    __shared__ Two scratch[33];
    __shared__ uint32_t s_bad, s_shared;
    __shared__ int32_t s_groups[kPlanThreads];
    __shared__ uint32_t s_bits[kPlanThreads];
    __shared__ int32_t s_rank[kPlanThreads];
    PagesHeader *head = p.s.head;
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = s_shared = 0;
    let_next_start();
    wait_for_inputs();
    // asked for now, needed after the lists are counted: the free counts and
    // the first group's words (a plan is a chain of memory latencies)
    const int32_t n_free = head->n_free;
    int32_t groups = tid < p.s.n_groups ? p.s.group_free[tid] : 0;
    const uint32_t bits0 = tid < p.s.n_words ? p.s.bitmap[tid] : 0;
    __syncthreads();
    uint32_t bad = 0;
    Two sum{0, 0};
    bool shares = false;
    ListPlan list{0, 0, -1};
    for (int base = 0; base < p.n_lists; base += kPlanThreads) {
        const int i = base + tid;
        Two need{0, 0}, all;
        if (i < p.n_lists) {
            need = list_needs(p, i, &bad, &list);
            shares |= list.shared >= 0;
            p.s.shared[i] = list.shared;
            p.s.old_len[i] = list.len;
        }
        const Two at = block_scan(need, scratch, &all);
        if (i < p.n_lists) {
            p.s.row_begin[i] = sum.rows + at.rows;
            p.s.page_begin[i] = (int32_t)(sum.pages + at.pages);
        }
        sum = sum + all;
        if (sum.pages > p.n_pages) {   // more than the pool holds
            if (tid == 0) atomicOr(&s_bad, KVC_DEV_PAGES_FULL);
            break;
        }
    }
    if (bad) atomicOr(&s_bad, bad);
    if (shares) s_shared = 1;
    __syncthreads();
    const uint32_t against = s_bad ? s_bad : sum.pages > n_free ? KVC_DEV_PAGES_FULL : 0;
    const bool ok = against == 0;
    if (tid == 0) {
        if (!ok) set_status(&head->status, against);
        head->ok = ok;
        head->total_new = (int32_t)sum.pages;
        head->total_rows = sum.rows;
        if (ok) {
            p.s.row_begin[p.n_lists] = sum.rows;
            p.s.page_begin[p.n_lists] = (int32_t)sum.pages;
        }
    }
    if (!ok) return;

    // the lowest free pages, group by group: each thread ranks a word of the
    // bitmap, then each writes down pages by rank
    const int need = (int)sum.pages;
    int found = 0;
    for (int g0 = 0; g0 < p.s.n_groups && found < need; g0 += kPlanThreads) {
        __syncthreads();
        if (g0 > 0) groups = g0 + tid < p.s.n_groups ? p.s.group_free[g0 + tid] : 0;
        s_groups[tid] = groups;
        __syncthreads();
        for (int j = 0; j < kPlanThreads && found < need; ++j) {
            if (s_groups[j] == 0) continue;
            const int word0 = (g0 + j) * kGroupWords, word = word0 + tid;
            const uint32_t bits = g0 + j == 0 ? bits0 : word < p.s.n_words ? p.s.bitmap[word] : 0;
            Two all;
            const int rank = (int)block_scan(Two{0, __popc(bits)}, scratch, &all).pages;
            const int took = min((int)all.pages, need - found);
            s_bits[tid] = bits;
            s_rank[tid] = rank;
            __syncthreads();
            for (int e = tid; e < took; e += kPlanThreads) {
                int lo = 0;
#pragma unroll
                for (int w = kPlanThreads / 2; w >= 1; w >>= 1)
                    if (s_rank[lo + w] <= e) lo += w;
                const int page = (word0 + lo) * 32 + nth_bit(s_bits[lo], e - s_rank[lo]);
                p.s.fresh[found + e] = page;
                p.s.holders[page] = 1;
            }
            if (rank < took && bits) {
                const int mine = min(__popc(bits), took - rank);
                p.s.bitmap[word] = mine == __popc(bits) ? 0 : bits & ~((2u << nth_bit(bits, mine - 1)) - 1u);
            }
            if (tid == 0) {
                p.s.group_free[g0 + j] = s_groups[j] - took;
                head->n_free = n_free - found - took;
            }
            found += took;
            __syncthreads();
        }
    }
    if (!p.append) return;
    // the lists' new lengths; their copied last pages lose a holder (after the
    // search, so that this call does not hand them out)
    __syncthreads();
    const bool drop = s_shared;
    for (int base = 0; base < p.n_lists; base += kPlanThreads) {
        const int i = base + tid;
        int32_t page = -1;
        if (i < p.n_lists) {
            if (p.n_lists > kPlanThreads) list = ListPlan{p.counts[i], p.s.old_len[i], p.s.shared[i]};
            page = list.shared;
            if (list.n > 0) p.len[i] = list.len + list.n;
        }
        if (drop) let_go(p.s, page, p.n_pages);
    }
}

struct MoveParams {
    PagesState s;
    int32_t *table;
    const int64_t *src_row;   // append: rows of the source
    int64_t src_step;
    const int32_t *idx;       // compact: rows of the list itself
    int32_t n_lists, n_pages, max_pages, shift, k_max;
    int vec;                  // 16-byte vectors per row
    Divider by_vec;
    const uint4 *k_src, *v_src;
    uint4 *k_pool, *v_pool;
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

template <bool APPEND>
__global__ void __launch_bounds__(kMoveThreads) pages_move_kernel(MoveParams p) {
    let_next_start();
    wait_for_inputs();
    if (!p.s.head->ok) return;
    const int64_t rows = p.s.head->total_rows;
    const int ps = 1 << p.shift, lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
    const int64_t me = ((int64_t)blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    if (APPEND) {   // the new pages' table entries, 32 a warp
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
    const int64_t per = (rows + warps - 1) / warps;
    const int64_t r0 = me * per, r1 = min(rows, r0 + per);
    if (r0 >= r1) return;
    int i = owner(p.s.row_begin, p.n_lists, r0);
    uint32_t bad = 0;
    const int items = (int)(r1 - r0) * p.vec;
    for (int it = lane; it < items; it += 32) {
        const int dr = p.by_vec(it), u = it - dr * p.vec;
        const int64_t r = r0 + dr;
        i = owner_from(p.s.row_begin, p.n_lists, r, i);
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
                    bad |= KVC_DEV_BAD_PAGE;
            } else {
                bad |= KVC_DEV_BAD_LIST;
            }
            to = ((int64_t)fresh[at >> p.shift] << p.shift) + (at & (ps - 1));
        }
        uint4 kk = make_uint4(0, 0, 0, 0), vv = kk;
        if (from >= 0) {
            kk = (own_pool ? p.k_pool : p.k_src)[from * p.vec + u];
            vv = (own_pool ? p.v_pool : p.v_src)[from * p.vec + u];
        }
        p.k_pool[to * p.vec + u] = kk;
        p.v_pool[to * p.vec + u] = vv;
    }
    if (!APPEND && bad) set_status(&p.s.head->status, bad);
}

// After a compaction's rows have moved: the lists take their new pages and let
// go of the old ones.
__global__ void __launch_bounds__(kListThreads)
    pages_swap_kernel(PagesState s, int32_t *table, int32_t *len, const int32_t *counts,
                      int32_t n_pages, int32_t max_pages, int shift) {
    let_next_start();
    wait_for_inputs();
    if (!s.head->ok) return;
    const int i = blockIdx.x;
    const int32_t n = counts[i];
    if (n < 0) return;
    const int ps = 1 << shift;
    const int had = (s.old_len[i] + ps - 1) >> shift, has = (n + ps - 1) >> shift;
    int32_t *entry = table + (int64_t)i * max_pages;
    const int32_t *fresh = s.fresh + s.page_begin[i];
    for (int j0 = 0; j0 < max(had, has); j0 += kListThreads) {
        const int j = j0 + threadIdx.x;
        int32_t old = -1;
        if (j < had) {
            old = entry[j];
            if (old < 0) set_status(&s.head->status, KVC_DEV_BAD_PAGE);
        }
        if (j < has) entry[j] = fresh[j];
        let_go(s, old, n_pages);
    }
    if (threadIdx.x == 0) len[i] = n;
}

__global__ void __launch_bounds__(kListThreads)
    pages_truncate_kernel(PagesState s, const int32_t *table, int32_t *len, const int32_t *new_len,
                          int32_t n_pages, int32_t max_pages, int shift) {
    const int i = blockIdx.x;
    let_next_start();
    wait_for_inputs();
    const int32_t want = new_len[i], now = len[i];
    const int ps = 1 << shift;
    __syncthreads();   // everyone has read len[i]
    if (want < 0) return;
    if (now < 0 || now > ((int64_t)max_pages << shift)) {
        if (threadIdx.x == 0) set_status(&s.head->status, KVC_DEV_BAD_LIST);
        return;
    }
    if (want >= now) return;
    const int had = (now + ps - 1) >> shift, has = (want + ps - 1) >> shift;
    for (int j0 = has; j0 < had; j0 += kListThreads) {
        const int j = j0 + threadIdx.x;
        int32_t old = -1;
        if (j < had) {
            old = table[(int64_t)i * max_pages + j];
            if (old < 0) set_status(&s.head->status, KVC_DEV_BAD_PAGE);
        }
        let_go(s, old, n_pages);
    }
    if (threadIdx.x == 0) len[i] = want;
}

__global__ void __launch_bounds__(kListThreads)
    pages_fork_kernel(PagesState s, int32_t *table, int32_t *len, const int32_t *src,
                      int32_t n_lists, int32_t n_pages, int32_t max_pages, int shift) {
    const int i = blockIdx.x;
    let_next_start();
    wait_for_inputs();
    const int32_t from = src[i];
    if (from < 0) return;
    const int ps = 1 << shift;
    const int32_t mine = len[i];
    __syncthreads();   // everyone has read len[i]
    // a source that this call forks into as well might be read half done
    const bool bad = from >= n_lists || mine != 0 || src[from] >= 0;
    const int32_t n = bad ? 0 : len[from];
    if (bad || n < 0 || n > ((int64_t)max_pages << shift)) {
        if (threadIdx.x == 0) set_status(&s.head->status, KVC_DEV_BAD_LIST);
        return;
    }
    const int held = (n + ps - 1) >> shift;
    for (int j = threadIdx.x; j < held; j += kListThreads) {
        const int32_t page = table[(int64_t)from * max_pages + j];
        table[(int64_t)i * max_pages + j] = page;
        if (page >= 0 && page < n_pages)
            atomicAdd(&s.holders[page], 1);
        else
            set_status(&s.head->status, KVC_DEV_BAD_PAGE);
    }
    if (threadIdx.x == 0) len[i] = n;
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

int launch_pages_init(const kvc_cache &c, const PagesState &s, cudaStream_t st) {
    pages_init_kernel<<<256, 256, 0, st>>>(s, c.n_pages);
    return cache_launched("kvc_pages_init");
}

int launch_pages_append(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                        int32_t n_lists, const int32_t *counts, const int64_t *src_row,
                        int64_t src_step, const void *k_src, const void *v_src, int64_t src_rows,
                        void *k_pool, void *v_pool, int sms, cudaStream_t st) {
    const int shift = log2_of(c.page_rows);
    PlanParams p{s, table, len, counts, src_row, src_step, src_rows, n_lists, c.n_pages, c.max_pages,
                 shift, 0, true};
    launch_early(pages_plan_kernel, 1, kPlanThreads, 0, st, p);
    const int vec = c.head_dim * (c.dtype == KVC_F32 ? 4 : 2) / 16;
    MoveParams m{s, table, src_row, src_step, nullptr, n_lists, c.n_pages, c.max_pages, shift, 0, vec, Divider(vec),
                 static_cast<const uint4 *>(k_src), static_cast<const uint4 *>(v_src),
                 static_cast<uint4 *>(k_pool), static_cast<uint4 *>(v_pool)};
    launch_early(pages_move_kernel<true>, sms * 8, kMoveThreads, 0, st, m);
    return cache_launched("kvc_pages_append");
}

int launch_pages_compact(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                         int32_t n_lists, const int32_t *idx, int32_t k_max, const int32_t *counts,
                         void *k_pool, void *v_pool, int sms, cudaStream_t st) {
    const int shift = log2_of(c.page_rows);
    PlanParams p{s, table, len, counts, nullptr, 0, 0, n_lists, c.n_pages, c.max_pages, shift, k_max,
                 false};
    launch_early(pages_plan_kernel, 1, kPlanThreads, 0, st, p);
    const int vec = c.head_dim * (c.dtype == KVC_F32 ? 4 : 2) / 16;
    MoveParams m{s, table, nullptr, 0, idx, n_lists, c.n_pages, c.max_pages, shift, k_max, vec, Divider(vec),
                 nullptr, nullptr, static_cast<uint4 *>(k_pool), static_cast<uint4 *>(v_pool)};
    launch_early(pages_move_kernel<false>, sms * 8, kMoveThreads, 0, st, m);
    launch_early(pages_swap_kernel, n_lists, kListThreads, 0, st, s, table, len, counts, c.n_pages,
                 c.max_pages, shift);
    return cache_launched("kvc_pages_compact");
}

int launch_pages_fork(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                      int32_t n_lists, const int32_t *src, cudaStream_t st) {
    launch_early(pages_fork_kernel, n_lists, kListThreads, 0, st, s, table, len, src, n_lists, c.n_pages,
                 c.max_pages, log2_of(c.page_rows));
    return cache_launched("kvc_pages_fork");
}

int launch_pages_truncate(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                          int32_t n_lists, const int32_t *new_len, cudaStream_t st) {
    launch_early(pages_truncate_kernel, n_lists, kListThreads, 0, st, s, table, len, new_len, c.n_pages,
                 c.max_pages, log2_of(c.page_rows));
    return cache_launched("kvc_pages_truncate");
}

}  // namespace kvc
