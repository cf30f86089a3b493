// cache.cuh -- what the paged-cache translation units share: the layout of the
// pages' state, the arguments of the launches, and device helpers that read a
// page table without trusting it.
#pragma once

#include <atomic>

#include "kvc_internal.cuh"

namespace kvc {

// ---------------------------------------------------------------- pages' state
// header | free pages per group | free bitmap | holders per page | page numbers
// of the running call | per-list scratch of the running call.  The three
// middle arrays say the same thing at three grains: holders[p] == 0 <=> bit p
// set, and a group's counter is its number of set bits, so that the search
// for free pages skips full stretches of a large pool.
constexpr int kGroupWords = 1024;                  // bitmap words of a group
constexpr int kGroupPages = 32 * kGroupWords;
constexpr size_t kPagesHeader = 256;
constexpr int kMaxLists = 1 << 20;

struct PagesHeader {
    uint32_t status;
    int32_t n_free;
    int32_t ok;          // whether the running call's plan stands
    int32_t total_new;   // pages it takes
    int64_t total_rows;  // rows it moves
};

struct PagesState {
    PagesHeader *head;
    int32_t *group_free;
    uint32_t *bitmap;
    int32_t *holders;
    int32_t *fresh;       // [n_pages] pages taken by the running call, ascending
    int64_t *row_begin;   // [n_lists + 1] rows moved for earlier lists
    int32_t *page_begin;  // [n_lists + 1] pages taken for earlier lists
    int32_t *old_len;     // [n_lists]
    int32_t *shared;      // [n_lists] last page to copy from, or -1
    int n_words, n_groups;
};

__host__ __device__ inline size_t cache_align(size_t x) { return (x + 255) & ~size_t(255); }

inline size_t pages_layout(const kvc_cache &c, int n_lists, char *base, PagesState *s) {
    PagesState t;
    t.n_words = (c.n_pages + 31) / 32;
    t.n_groups = (t.n_words + kGroupWords - 1) / kGroupWords;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = base + at;
        at += cache_align(bytes);
        return p;
    };
    t.head = reinterpret_cast<PagesHeader *>(take(kPagesHeader));
    t.group_free = reinterpret_cast<int32_t *>(take((size_t)t.n_groups * 4));
    t.bitmap = reinterpret_cast<uint32_t *>(take((size_t)t.n_words * 4));
    t.holders = reinterpret_cast<int32_t *>(take((size_t)c.n_pages * 4));
    t.fresh = reinterpret_cast<int32_t *>(take((size_t)c.n_pages * 4));
    t.row_begin = reinterpret_cast<int64_t *>(take(((size_t)n_lists + 1) * 8));
    t.page_begin = reinterpret_cast<int32_t *>(take(((size_t)n_lists + 1) * 4));
    t.old_len = reinterpret_cast<int32_t *>(take((size_t)n_lists * 4));
    t.shared = reinterpret_cast<int32_t *>(take((size_t)n_lists * 4));
    if (s) *s = t;
    return at;
}

// ---------------------------------------------------------------- launches
struct RopeArgs {
    int32_t dtype;
    int64_t n_tokens;
    int32_t n_q_heads, n_k_heads, head_dim, rot_dim;
    uint32_t flags;
    float amplitude;
    const int32_t *positions;
    const uint64_t *table;
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, q_out_stride, k_stride, k_out_stride;
};

// n / d for n < 2^31 by a multiplication and a shift (the round-up method of
// Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): the walk over units divides a lot.
struct Divider {
    uint32_t d, mul, shift;
    __host__ __device__ Divider() {}
    explicit Divider(uint32_t by) : d(by), shift(0) {
        while (((uint64_t)1 << shift) < by) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ int operator()(int n) const {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
};

// Launches of these operators may begin before the kernel in front has ended
// (programmatic dependent launch): a kernel waits with wait_for_inputs() before
// it touches memory, which ends when everything in front is complete and
// visible, and only its launch latency is hidden.  let_next_start() says that
// the next kernel's blocks may be brought in.
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Lets a kernel use up to `bytes` of shared memory per block; asked of the driver
// once per kernel and device.
template <auto kKernel>
void allow_shared(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return;   // the launch will say so
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
}

template <typename... P, typename... A>
void launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, P(args)...);   // errors stay for cache_launched
}

// KVC_OK, or KVC_ERR_CUDA with a message if the launches before failed.
int cache_launched(const char *fn);

int launch_rope_table(int32_t rot, double theta, double factor, double alpha, double beta,
                      double context, uint64_t *table, cudaStream_t st);
int launch_rope(const RopeArgs &a, int sms, cudaStream_t st);

int launch_pages_init(const kvc_cache &c, const PagesState &s, cudaStream_t st);
int launch_pages_append(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                        int32_t n_lists, const int32_t *counts, const int64_t *src_row,
                        int64_t src_step, const void *k_src, const void *v_src, int64_t src_rows,
                        void *k_pool, void *v_pool, int sms, cudaStream_t st);
int launch_pages_fork(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                      int32_t n_lists, const int32_t *src, cudaStream_t st);
int launch_pages_compact(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                         int32_t n_lists, const int32_t *idx, int32_t k_max, const int32_t *counts,
                         void *k_pool, void *v_pool, int sms, cudaStream_t st);
int launch_pages_truncate(const kvc_cache &c, const PagesState &s, int32_t *table, int32_t *len,
                          int32_t n_lists, const int32_t *new_len, cudaStream_t st);

}  // namespace kvc
