// api_cache.cu -- the extern "C" entry points of the paged cache: argument
// validation, the layout of the pages' state and of the attention's workspace,
// and dispatch to the kernels.  As in api.cu, nothing here allocates device
// memory and every launch goes to the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "attend.cuh"
#include "quant.cuh"

namespace kvc {

namespace {

template <typename... A>
int fail(int code, const char *fmt, A... a) {
    set_error(fmt, a...);
    return code;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int device_sms() {
    static std::mutex mu;
    static int cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0 &&
        cudaDeviceGetAttribute(&cache[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        cudaGetLastError();
    return cache[dev];
}

bool cache_ok(const kvc_cache *c, const char *fn) {
    if (!c) return fail(0, "%s: cache is NULL", fn), false;
    if (c->n_pages < 1 || c->n_pages > (1 << 30))
        return fail(0, "%s: n_pages must be in 1..2^30", fn), false;
    if (c->page_rows != 16 && c->page_rows != 32 && c->page_rows != 64 && c->page_rows != 128)
        return fail(0, "%s: page_rows must be 16, 32, 64 or 128", fn), false;
    if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8)
        return fail(0, "%s: head_dim must be a multiple of 8 in 8..256", fn), false;
    if (c->dtype != KVC_F32 && c->dtype != KVC_BF16)
        return fail(0, "%s: unknown dtype %d", fn, c->dtype), false;
    // 256 short of 2^31, so that the end of a list's last step is still an int
    if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_rows > ((int64_t)1 << 31) - 256)
        return fail(0, "%s: max_pages must be >= 1 and max_pages * page_rows <= 2^31 - 256", fn), false;
    return true;
}

bool bits_ok(int32_t bits, const char *fn) {
    if (bits != 4 && bits != 8) return fail(0, "%s: bits must be 4 or 8", fn), false;
    return true;
}

bool lists_ok(int32_t n_lists, const char *fn) {
    if (n_lists < 1 || n_lists > kMaxLists)
        return fail(0, "%s: n_lists must be in 1..2^20", fn), false;
    return true;
}

// The state of a call over n_lists lists, or an error code.
int state_of(const kvc_cache &c, int32_t n_lists, void *state, size_t bytes, const char *fn,
             PagesState *s) {
    if (!state) return fail(KVC_ERR_WORKSPACE, "%s: state is NULL", fn);
    if (reinterpret_cast<uintptr_t>(state) % 256)
        return fail(KVC_ERR_WORKSPACE, "%s: state must be 256-byte aligned", fn);
    const size_t need = pages_layout(c, n_lists, static_cast<char *>(state), s);
    if (bytes < need)
        return fail(KVC_ERR_WORKSPACE, "%s: state has %zu bytes, needs %zu", fn, bytes, need);
    return KVC_OK;
}

// The kernel that takes a call, and its workspace: header | arrival counters |
// slots' (max, sum) | groups' (max, sum) | slots' rows.
struct AttendWs {
    bool tc;
    AttendNeeds needs;
    size_t arrived, stat, group_stat, part, total;
};

AttendWs attend_ws(const kvc_cache &c, int group) {
    AttendWs w;
    w.tc = attend_tc_takes(c.dtype, c.head_dim, group);
    w.needs = w.tc ? attend_tc_needs(device_sms()) : attend_simt_needs(device_sms());
    const size_t rows = (size_t)w.needs.grid * w.needs.slots * w.needs.slot_rows;
    w.arrived = kWsHeader;
    // as many counters for either kernel: one's scratch is never the other's
    // counters, so a workspace may serve caches of several kinds
    const int counters = 16 * std::max(attend_tc_needs(device_sms()).grid, attend_simt_needs(device_sms()).grid);
    w.stat = w.arrived + cache_align((size_t)counters * sizeof(uint32_t));
    w.group_stat = w.stat + cache_align(rows * sizeof(float2));
    w.part = w.group_stat + cache_align(rows * sizeof(float2));
    w.total = w.part + cache_align(rows * c.head_dim * sizeof(float));
    return w;
}

bool attend_shape_ok(const kvc_cache *c, int32_t n_q_heads, int32_t n_kv_heads, int32_t n_seqs,
                     int32_t max_new, const char *fn) {
    if (!cache_ok(c, fn)) return false;
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads)
        return fail(0, "%s: n_q_heads must be a positive multiple of n_kv_heads", fn), false;
    if (n_seqs < 1 || (int64_t)n_seqs * n_kv_heads > kMaxLists)
        return fail(0, "%s: n_seqs * n_kv_heads must be in 1..2^20", fn), false;
    if (max_new < 1 || (int64_t)max_new * (n_q_heads / n_kv_heads) > (1 << 30))
        return fail(0, "%s: max_new must be >= 1 and max_new * query heads per KV head <= 2^30", fn), false;
    return true;
}

// kvc_attend and kvc_attend_quant; bits 0: rows of the cache's own type.
int attend_call(const char *fn, int bits, const kvc_cache *cache, int32_t n_q_heads, int32_t n_kv_heads,
                int32_t n_seqs, int32_t max_new, int64_t n_tokens, const void *q, int64_t q_stride,
                const int32_t *q_start, const int32_t *table, const int32_t *len, const void *k_pool,
                const void *v_pool, float scale, void *out, float *lse, uint32_t flags, void *ws, size_t ws_bytes,
                cudaStream_t stream) {
    set_error("%s", "");
    if (flags & ~KVC_ATTEND_BF16_P) return fail(KVC_ERR_INVALID_ARG, "%s: unknown flags %#x", fn, flags);
    if (!attend_shape_ok(cache, n_q_heads, n_kv_heads, n_seqs, max_new, fn))
        return KVC_ERR_INVALID_ARG;
    const kvc_cache &c = *cache;
    if (n_tokens < 0 || n_tokens >= ((int64_t)1 << 31))
        return fail(KVC_ERR_INVALID_ARG, "%s: n_tokens must be in 0..2^31-1", fn);
    if (n_tokens == 0) return KVC_OK;   // empty tensors have no address
    if (!q || !q_start || !table || !len || !k_pool || !v_pool || !out)
        return fail(KVC_ERR_INVALID_ARG, "%s: NULL tensor", fn);
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
        return fail(KVC_ERR_INVALID_ARG, "%s: q, out and pools must be 16-byte aligned", fn);
    if (q_stride < (int64_t)n_q_heads * c.head_dim || q_stride % 8 || q_stride > ((int64_t)1 << 38))
        return fail(KVC_ERR_INVALID_ARG,
                    "%s: q_stride must be a multiple of 8 and >= n_q_heads * head_dim", fn);
    if (!std::isfinite((float)(scale * kLog2e)))
        return fail(KVC_ERR_INVALID_ARG, "%s: scale must be finite (times log2 e, too)", fn);
    const AttendWs w = attend_ws(c, n_q_heads / n_kv_heads);
    if (w.needs.grid == 0) return fail(KVC_ERR_CUDA, "%s: no usable CUDA device", fn);
    if (!ws) return fail(KVC_ERR_WORKSPACE, "%s: workspace is NULL", fn);
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return fail(KVC_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
    if (ws_bytes < w.total)
        return fail(KVC_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws_bytes, w.total);
    char *base = static_cast<char *>(ws);
    AttendParams p{};
    p.n_seqs = n_seqs;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_q_heads / n_kv_heads;
    p.dim = c.head_dim;
    p.bits = bits;
    p.n_pages = c.n_pages;
    p.max_pages = c.max_pages;
    while ((1 << p.shift) < c.page_rows) ++p.shift;
    p.n_tokens = n_tokens;
    p.max_new = max_new;
    p.slots = w.needs.slots;
    p.slot_rows = w.needs.slot_rows;
    p.q_stride = q_stride;
    p.q = q;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.q_start = q_start;
    p.table = table;
    p.len = len;
    p.out = out;
    p.lse = lse;
    p.scale_log2 = (float)(scale * kLog2e);
    p.one_term = flags & KVC_ATTEND_BF16_P;
    p.status = static_cast<uint32_t *>(ws);
    p.arrived = reinterpret_cast<uint32_t *>(base + w.arrived);
    p.stat = reinterpret_cast<float2 *>(base + w.stat);
    p.group_stat = reinterpret_cast<float2 *>(base + w.group_stat);
    p.part = reinterpret_cast<float *>(base + w.part);
    const bool f32 = c.dtype == KVC_F32;
    if (bits != 0 && w.tc) {
        // Lists of few rows are attend_quant.cu's: a tile of tcgen05's is 128 rows whoever
        // fills them, and its keys are written out as bf16 first (us here and there; 64 x 8
        // lists of 500-6,000 rows of 128 in 4 bits: 4 rows a list 82 and 299, 16 rows 120
        // and 301, 32 rows 225 and 308; 32 x 8 in 8 bits: 58 and 198, 75 and 202, 130 and
        // 214; heads of 64, 64 x 8 lists, 32 rows: 126 and 199, in 8 bits 128 and 207; one
        // sequence of 1,000: 12 and 19).  48 rows would be three units of 16, where two take
        // 225, and are 317 there.
        // Where chunks are among them, a token's rows go in a launch of their own as in
        // launch_attend_simt, unless a token has more.
        const int few = attend_quant_rows();
        const int64_t most = (int64_t)max_new * p.group;
        if (most <= few) return launch_attend_quant(p, (int)most, w.needs.grid, stream);
        const int own = p.group <= 8 ? 8 : p.group <= 16 ? 16 : 32;
        const bool both = p.group <= few && n_tokens * p.group <= 128 * (int64_t)n_seqs;
        // (the one that may be refused comes first: then nothing has been written)
        const int rc = launch_attend_tc_quant(p, both ? own : 0, w.needs.grid, stream);
        return rc || !both ? rc : launch_attend_quant(p, own, w.needs.grid, stream);
    }
    if (bits != 0)
        return bits == 4 ? launch_attend_simt_quant4(p, f32, w.needs.grid, stream)
                         : launch_attend_simt_quant8(p, f32, w.needs.grid, stream);
    return w.tc ? launch_attend_tc(p, w.needs.grid, stream) : launch_attend_simt(p, f32, w.needs.grid, stream);
}

}  // namespace

int cache_launched(const char *fn) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(KVC_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    return KVC_OK;
}

}  // namespace kvc

using namespace kvc;

extern "C" {

size_t kvc_pages_size(const kvc_cache *cache, int32_t n_lists) {
    if (!cache_ok(cache, "kvc_pages_size") || !lists_ok(n_lists, "kvc_pages_size")) return 0;
    return pages_layout(*cache, n_lists, nullptr, nullptr);
}

int kvc_pages_init(const kvc_cache *cache, void *state, size_t state_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_init");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_init")) return KVC_ERR_INVALID_ARG;
    PagesState s;
    const int rc = state_of(*cache, 1, state, state_bytes, "kvc_pages_init", &s);
    return rc ? rc : launch_pages_init(*cache, s, stream);
}

int kvc_pages_status(const kvc_cache *cache, const void *state, size_t state_bytes,
                     uint32_t *status, int32_t *n_free, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_status");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_status")) return KVC_ERR_INVALID_ARG;
    PagesState s;
    const int rc = state_of(*cache, 1, const_cast<void *>(state), state_bytes, "kvc_pages_status", &s);
    if (rc) return rc;
    PagesHeader h;
    cudaError_t e = cudaMemcpyAsync(&h, s.head, sizeof h, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return fail(KVC_ERR_CUDA, "kvc_pages_status: %s", cudaGetErrorString(e));
    if (status) *status = h.status;
    if (n_free) *n_free = h.n_free;
    return KVC_OK;
}

int kvc_pages_append(const kvc_cache *cache, int32_t *table, int32_t *len, int32_t n_lists,
                     const int32_t *counts, const int64_t *src_row, int64_t src_step,
                     const void *k_src, const void *v_src, int64_t src_rows, void *k_pool,
                     void *v_pool, void *state, size_t state_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_append");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_append") || !lists_ok(n_lists, "kvc_pages_append"))
        return KVC_ERR_INVALID_ARG;
    if (!table || !len || !counts || !src_row || (src_rows != 0 && (!k_src || !v_src)) || !k_pool || !v_pool)
        return fail(KVC_ERR_INVALID_ARG, "kvc_pages_append: NULL tensor");
    if (!aligned16(k_src) || !aligned16(v_src) || !aligned16(k_pool) || !aligned16(v_pool))
        return fail(KVC_ERR_INVALID_ARG, "kvc_pages_append: rows and pools must be 16-byte aligned");
    if (src_step < 0 || src_rows < 0)
        return fail(KVC_ERR_INVALID_ARG, "kvc_pages_append: src_step and src_rows must be >= 0");
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, "kvc_pages_append", &s);
    if (rc) return rc;
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "kvc_pages_append: no usable CUDA device");
    return launch_pages_append(*cache, s, table, len, n_lists, counts, src_row, src_step, k_src, v_src,
                               src_rows, k_pool, v_pool, sms, stream);
}

int kvc_pages_fork(const kvc_cache *cache, int32_t *table, int32_t *len, int32_t n_lists,
                   const int32_t *src, void *state, size_t state_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_fork");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_fork") || !lists_ok(n_lists, "kvc_pages_fork"))
        return KVC_ERR_INVALID_ARG;
    if (!table || !len || !src) return fail(KVC_ERR_INVALID_ARG, "kvc_pages_fork: NULL tensor");
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, "kvc_pages_fork", &s);
    return rc ? rc : launch_pages_fork(*cache, s, table, len, n_lists, src, stream);
}

int kvc_pages_compact(const kvc_cache *cache, int32_t *table, int32_t *len, int32_t n_lists,
                      const int32_t *idx, int32_t k_max, const int32_t *counts, void *k_pool,
                      void *v_pool, void *state, size_t state_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_compact");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_compact") || !lists_ok(n_lists, "kvc_pages_compact"))
        return KVC_ERR_INVALID_ARG;
    if (!table || !len || !idx || !counts || !k_pool || !v_pool)
        return fail(KVC_ERR_INVALID_ARG, "kvc_pages_compact: NULL tensor");
    if (k_max < 1) return fail(KVC_ERR_INVALID_ARG, "kvc_pages_compact: k_max must be >= 1");
    if (!aligned16(k_pool) || !aligned16(v_pool))
        return fail(KVC_ERR_INVALID_ARG, "kvc_pages_compact: pools must be 16-byte aligned");
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, "kvc_pages_compact", &s);
    if (rc) return rc;
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "kvc_pages_compact: no usable CUDA device");
    return launch_pages_compact(*cache, s, table, len, n_lists, idx, k_max, counts, k_pool, v_pool, sms,
                                stream);
}

int kvc_pages_truncate(const kvc_cache *cache, int32_t *table, int32_t *len, int32_t n_lists,
                       const int32_t *new_len, void *state, size_t state_bytes,
                       cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_pages_truncate");
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_pages_truncate") || !lists_ok(n_lists, "kvc_pages_truncate"))
        return KVC_ERR_INVALID_ARG;
    if (!table || !len || !new_len) return fail(KVC_ERR_INVALID_ARG, "kvc_pages_truncate: NULL tensor");
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, "kvc_pages_truncate", &s);
    return rc ? rc : launch_pages_truncate(*cache, s, table, len, n_lists, new_len, stream);
}

int kvc_rope_table(int32_t rot_dim, double theta, double factor, double alpha, double beta,
                   double context, uint64_t *table, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_rope_table");
    set_error("%s", "");
    if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2)
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope_table: rot_dim must be even, 2..256");
    if (!(theta >= 1.0) || std::isinf(theta))
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope_table: theta must be >= 1 and finite");
    if (!(factor >= 1.0) || std::isinf(factor))
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope_table: factor must be >= 1 and finite");
    if (factor > 1.0 && (!(alpha >= 0.0) || !(beta >= alpha) || !(context > 0.0) || std::isinf(context)))
        return fail(KVC_ERR_INVALID_ARG,
                    "kvc_rope_table: need 0 <= alpha <= beta and a positive, finite context");
    if (!table || reinterpret_cast<uintptr_t>(table) % 8)
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope_table: table must be an 8-byte aligned tensor");
    return launch_rope_table(rot_dim, theta, factor, alpha, beta, context, table, stream);
}

int kvc_rope(int32_t dtype, int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
             int32_t head_dim, int32_t rot_dim, uint32_t flags, float amplitude,
             const int32_t *positions, const uint64_t *table, const void *q, int64_t q_stride,
             void *q_out, int64_t q_out_stride, const void *k, int64_t k_stride, void *k_out,
             int64_t k_out_stride, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_rope");
    set_error("%s", "");
    if (dtype != KVC_F32 && dtype != KVC_BF16)
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope: unknown dtype %d", dtype);
    if (n_tokens < 0 || n_tokens >= ((int64_t)1 << 31))
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope: n_tokens must be in 0..2^31-1");
    if (head_dim < 2 || head_dim > 256 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope: need an even rot_dim in 2..head_dim and head_dim <= 256");
    if (flags & ~(KVC_ROPE_INTERLEAVED | KVC_ROPE_INVERSE))
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope: unknown flags %#x", flags);
    if (n_q_heads < 0 || n_k_heads < 0 || n_q_heads > (1 << 16) || n_k_heads > (1 << 16) ||
        n_q_heads + n_k_heads == 0)
        return fail(KVC_ERR_INVALID_ARG, "kvc_rope: heads must be in 0..65536, one at least");
    if (n_tokens == 0) return KVC_OK;   // empty tensors have no address
    if (!positions || !table) return fail(KVC_ERR_INVALID_ARG, "kvc_rope: NULL positions or table");
    struct {
        const char *name;
        int32_t heads;
        const void *x, *y;
        int64_t xs, ys;
    } sides[2] = {{"q", n_q_heads, q, q_out, q_stride, q_out_stride},
                  {"k", n_k_heads, k, k_out, k_stride, k_out_stride}};
    const uintptr_t es = dtype == KVC_F32 ? 4 : 2;
    for (const auto &s : sides) {
        if (s.heads == 0) continue;
        if (!s.x || !s.y) return fail(KVC_ERR_INVALID_ARG, "kvc_rope: NULL %s tensor", s.name);
        if (reinterpret_cast<uintptr_t>(s.x) % es || reinterpret_cast<uintptr_t>(s.y) % es)
            return fail(KVC_ERR_INVALID_ARG, "kvc_rope: %s is not aligned to its type", s.name);
        const int64_t row = (int64_t)s.heads * head_dim;
        if (s.xs < row || s.ys < row)
            return fail(KVC_ERR_INVALID_ARG, "kvc_rope: %s strides must be >= heads * head_dim", s.name);
        if (s.x == s.y && s.xs != s.ys)
            return fail(KVC_ERR_INVALID_ARG, "kvc_rope: %s in place needs one stride", s.name);
    }
    const RopeArgs a{dtype, n_tokens, n_q_heads, n_k_heads, head_dim, rot_dim, flags, amplitude, positions,
                     table, q, k, q_out, k_out, q_stride, q_out_stride, k_stride, k_out_stride};
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "kvc_rope: no usable CUDA device");
    return launch_rope(a, sms, stream);
}

size_t kvc_attend_workspace_size(const kvc_cache *cache, int32_t n_q_heads, int32_t n_kv_heads,
                                 int32_t n_seqs, int32_t max_new) {
    if (!attend_shape_ok(cache, n_q_heads, n_kv_heads, n_seqs, max_new, "kvc_attend_workspace_size"))
        return 0;
    return attend_ws(*cache, n_q_heads / n_kv_heads).total;
}

int kvc_attend(const kvc_cache *cache, int32_t n_q_heads, int32_t n_kv_heads, int32_t n_seqs,
               int32_t max_new, int64_t n_tokens, const void *q, int64_t q_stride,
               const int32_t *q_start, const int32_t *table, const int32_t *len,
               const void *k_pool, const void *v_pool, float scale, void *out, float *lse,
               void *ws, size_t ws_bytes, cudaStream_t stream) {
    return kvc_attend_ex(cache, n_q_heads, n_kv_heads, n_seqs, max_new, n_tokens, q, q_stride, q_start, table,
                         len, k_pool, v_pool, scale, out, lse, 0, ws, ws_bytes, stream);
}

int kvc_attend_ex(const kvc_cache *cache, int32_t n_q_heads, int32_t n_kv_heads, int32_t n_seqs,
                  int32_t max_new, int64_t n_tokens, const void *q, int64_t q_stride,
                  const int32_t *q_start, const int32_t *table, const int32_t *len,
                  const void *k_pool, const void *v_pool, float scale, void *out, float *lse,
                  uint32_t flags, void *ws, size_t ws_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("kvc_attend");
    return attend_call("kvc_attend", 0, cache, n_q_heads, n_kv_heads, n_seqs, max_new, n_tokens, q, q_stride, q_start,
                       table, len, k_pool, v_pool, scale, out, lse, flags, ws, ws_bytes, stream);
}

size_t kvc_quant_page_size(const kvc_cache *cache, int32_t bits) {
    set_error("%s", "");
    if (!cache_ok(cache, "kvc_quant_page_size") || !bits_ok(bits, "kvc_quant_page_size")) return 0;
    return (size_t)(cache->page_rows / kQuantRows) * quant_block(bits, quant_groups(cache->head_dim));
}

int kvc_pages_append_quant(const kvc_cache *cache, int32_t bits, int32_t *table, int32_t *len, int32_t n_lists,
                           const int32_t *counts, const int64_t *src_row, int64_t src_step, const void *k_src,
                           const void *v_src, int64_t src_rows, void *k_pool, void *v_pool, void *state,
                           size_t state_bytes, cudaStream_t stream) {
    const char *fn = "kvc_pages_append_quant";
    NvtxRange nvtx_range(fn);
    set_error("%s", "");
    if (!cache_ok(cache, fn) || !bits_ok(bits, fn) || !lists_ok(n_lists, fn)) return KVC_ERR_INVALID_ARG;
    if (!table || !len || !counts || !src_row || (src_rows != 0 && (!k_src || !v_src)) || !k_pool || !v_pool)
        return fail(KVC_ERR_INVALID_ARG, "%s: NULL tensor", fn);
    if (!aligned16(k_src) || !aligned16(v_src) || !aligned16(k_pool) || !aligned16(v_pool))
        return fail(KVC_ERR_INVALID_ARG, "%s: rows and pools must be 16-byte aligned", fn);
    if (src_step < 0 || src_rows < 0)
        return fail(KVC_ERR_INVALID_ARG, "%s: src_step and src_rows must be >= 0", fn);
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, fn, &s);
    if (rc) return rc;
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "%s: no usable CUDA device", fn);
    return launch_pages_append_quant(*cache, bits, s, table, len, n_lists, counts, src_row, src_step, k_src, v_src,
                                     src_rows, k_pool, v_pool, sms, stream);
}

int kvc_pages_compact_quant(const kvc_cache *cache, int32_t bits, int32_t *table, int32_t *len, int32_t n_lists,
                            const int32_t *idx, int32_t k_max, const int32_t *counts, void *k_pool, void *v_pool,
                            void *state, size_t state_bytes, cudaStream_t stream) {
    const char *fn = "kvc_pages_compact_quant";
    NvtxRange nvtx_range(fn);
    set_error("%s", "");
    if (!cache_ok(cache, fn) || !bits_ok(bits, fn) || !lists_ok(n_lists, fn)) return KVC_ERR_INVALID_ARG;
    if (!table || !len || !idx || !counts || !k_pool || !v_pool)
        return fail(KVC_ERR_INVALID_ARG, "%s: NULL tensor", fn);
    if (k_max < 1) return fail(KVC_ERR_INVALID_ARG, "%s: k_max must be >= 1", fn);
    if (!aligned16(k_pool) || !aligned16(v_pool))
        return fail(KVC_ERR_INVALID_ARG, "%s: pools must be 16-byte aligned", fn);
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, fn, &s);
    if (rc) return rc;
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "%s: no usable CUDA device", fn);
    return launch_pages_compact_quant(*cache, bits, s, table, len, n_lists, idx, k_max, counts, k_pool, v_pool, sms,
                                      stream);
}

int kvc_pages_read_quant(const kvc_cache *cache, int32_t bits, const int32_t *table, const int32_t *len,
                         int32_t n_lists, const int32_t *first, const int32_t *counts, const int64_t *dst_row,
                         int64_t dst_step, const void *k_pool, const void *v_pool, void *k_dst, void *v_dst,
                         int64_t dst_rows, void *state, size_t state_bytes, cudaStream_t stream) {
    const char *fn = "kvc_pages_read_quant";
    NvtxRange nvtx_range(fn);
    set_error("%s", "");
    if (!cache_ok(cache, fn) || !bits_ok(bits, fn) || !lists_ok(n_lists, fn)) return KVC_ERR_INVALID_ARG;
    if (!table || !len || !counts || !dst_row || (k_dst && !k_pool) || (v_dst && !v_pool) ||
        (dst_rows != 0 && !k_dst && !v_dst))
        return fail(KVC_ERR_INVALID_ARG, "%s: NULL tensor", fn);
    if (!aligned16(k_dst) || !aligned16(v_dst) || !aligned16(k_pool) || !aligned16(v_pool))
        return fail(KVC_ERR_INVALID_ARG, "%s: rows and pools must be 16-byte aligned", fn);
    if (dst_step < 0 || dst_rows < 0)
        return fail(KVC_ERR_INVALID_ARG, "%s: dst_step and dst_rows must be >= 0", fn);
    PagesState s;
    const int rc = state_of(*cache, n_lists, state, state_bytes, fn, &s);
    if (rc) return rc;
    const int sms = device_sms();
    if (sms == 0) return fail(KVC_ERR_CUDA, "%s: no usable CUDA device", fn);
    return launch_pages_read_quant(*cache, bits, s, table, len, n_lists, first, counts, dst_row, dst_step, k_pool,
                                   v_pool, k_dst, v_dst, dst_rows, sms, stream);
}

size_t kvc_attend_quant_workspace_size(const kvc_cache *cache, int32_t bits, int32_t n_q_heads, int32_t n_kv_heads,
                                       int32_t n_seqs, int32_t max_new) {
    const char *fn = "kvc_attend_quant_workspace_size";
    if (!attend_shape_ok(cache, n_q_heads, n_kv_heads, n_seqs, max_new, fn) || !bits_ok(bits, fn)) return 0;
    return attend_ws(*cache, n_q_heads / n_kv_heads).total;
}

int kvc_attend_quant(const kvc_cache *cache, int32_t bits, int32_t n_q_heads, int32_t n_kv_heads, int32_t n_seqs,
                     int32_t max_new, int64_t n_tokens, const void *q, int64_t q_stride, const int32_t *q_start,
                     const int32_t *table, const int32_t *len, const void *k_pool, const void *v_pool, float scale,
                     void *out, float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    return kvc_attend_quant_ex(cache, bits, n_q_heads, n_kv_heads, n_seqs, max_new, n_tokens, q, q_stride, q_start,
                               table, len, k_pool, v_pool, scale, out, lse, 0, ws, ws_bytes, stream);
}

int kvc_attend_quant_ex(const kvc_cache *cache, int32_t bits, int32_t n_q_heads, int32_t n_kv_heads, int32_t n_seqs,
                        int32_t max_new, int64_t n_tokens, const void *q, int64_t q_stride, const int32_t *q_start,
                        const int32_t *table, const int32_t *len, const void *k_pool, const void *v_pool, float scale,
                        void *out, float *lse, uint32_t flags, void *ws, size_t ws_bytes, cudaStream_t stream) {
    const char *fn = "kvc_attend_quant";
    NvtxRange nvtx_range(fn);
    if (!bits_ok(bits, fn)) return KVC_ERR_INVALID_ARG;
    return attend_call(fn, bits, cache, n_q_heads, n_kv_heads, n_seqs, max_new, n_tokens, q, q_stride, q_start, table,
                       len, k_pool, v_pool, scale, out, lse, flags, ws, ws_bytes, stream);
}

}  // extern "C"
