// attend.cuh -- the work split and the joining of partial results that both
// attention kernels (attend_simt.cu, attend_tc.cu) share.
//
// Rows: the G query heads of a KV head stand side by side, row r of a list =
// token r / G, query head r % G of the group, so every key tile is read once
// for all of them.  A unit is (list, block of unit_rows rows); its cost is
// its number of steps over the keys its last row sees (one at least, so that
// somebody writes the zeros of a row that sees none) and `extra` for what a unit
// costs beside them.  The flat sequence of all units' costs is cut into equal
// runs, one per CTA: lists of any lengths keep every SM busy to the end, and a CTA shares at most its first and its last
// unit with others.  For those it leaves rows' (max, sum, unnormalised output)
// in a slot of its own; the CTA that finishes last adds the unit's slots up in
// CTA order (of many slots, neighbours first), so the result does not depend on
// the order of finishing.
#pragma once

#include <algorithm>
#include <climits>

#include "cache.cuh"

namespace kvc {

struct AttendParams {
    int n_seqs, n_q_heads, n_kv_heads, group, dim;
    Divider by_group, by_heads, by_blocks;
    int n_pages, max_pages, shift;
    int64_t n_tokens;
    int max_new;
    int unit_rows;       // rows of a unit
    int blocks;          // units per list
    int n_units;
    int step_keys;       // keys per step ...
    int split_rows;      // ... twice as many for units of at most so many rows
    int rows_above, rows_upto;   // lists of so many rows are this launch's
    int extra;           // steps' worth of a unit's beginning and end
    int slots;           // slots per CTA
    int slot_rows;       // row capacity of a slot
    int64_t q_stride;
    const void *q, *k_pool, *v_pool;
    const int32_t *q_start, *table, *len;
    void *out;
    float *lse;
    float scale_log2;    // scale * log2(e)
    int skip_load;       // tests: every CTA's first load is left out
    bool one_term;       // tensor cores: probabilities in one bf16 term, not two
    uint32_t *status;
    Divider by_quads;    // dim / 4
    uint32_t *arrived;   // [grid][2][8], zero between calls: of a unit, of a group
    float2 *stat;        // [grid][slots][slot_rows] (max in log2 units, sum)
    float2 *group_stat;  // the same of joined groups
    float *part;         // [grid][slots][slot_rows][dim]
};

struct AttendUnit {
    int list, b, h;
    int q0, n;        // the sequence's first token and number of tokens
    int row0, rows;   // this unit's rows among the list's n * group
    int len;          // the list's cached rows
    int hi;           // cached rows that the unit's last row sees
    int steps;        // 0: no such unit
    int cost;         // steps + extra, or 0
};

// What a unit is made of in memory, to be asked for before it is needed.
struct AttendRaw {
    int q0, q1, len;
};
__device__ __forceinline__ AttendRaw attend_raw(const AttendParams &p, int u) {
    if (u >= p.n_units) return AttendRaw{0, 0, 0};
    const int list = p.by_blocks(u), b = p.by_heads(list);
    return AttendRaw{p.q_start[b], p.q_start[b + 1], p.len[list]};
}

// kSome: the launch has only lists of so many rows.
template <bool kSome>
__device__ __forceinline__ AttendUnit attend_unit(const AttendParams &p, int u, const AttendRaw &raw) {
    AttendUnit a;
    a.list = p.by_blocks(u);
    const int block = u - a.list * p.blocks;
    a.b = p.by_heads(a.list);
    a.h = a.list - a.b * p.n_kv_heads;
    int q0 = raw.q0, q1 = raw.q1;
    a.len = raw.len;
    const int64_t most = (int64_t)p.max_pages << p.shift;
    if (q0 < 0 || q1 < q0 || q1 > p.n_tokens || q1 - q0 > p.max_new || a.len < 0 || a.len > most) {
        set_status(p.status, KVC_DEV_BAD_LIST);
        q0 = max(q0, 0);
        q1 = (int)min((int64_t)min(q1, q0 > INT_MAX - p.max_new ? INT_MAX : q0 + p.max_new), p.n_tokens);
        a.len = (int)max((int64_t)0, min((int64_t)a.len, most));
    }
    a.q0 = q0;
    a.n = max(0, q1 - q0);
    if (kSome && (a.n * p.group <= p.rows_above || a.n * p.group > p.rows_upto)) a.n = 0;
    a.row0 = block * p.unit_rows;
    a.rows = min(p.unit_rows, a.n * p.group - a.row0);
    a.hi = a.rows <= 0 ? 0 : max(0, a.len - a.n + p.by_group(a.row0 + a.rows - 1) + 1);
    const int keys = a.rows <= p.split_rows ? 2 * p.step_keys : p.step_keys;
    a.steps = a.rows <= 0 ? 0 : max(1, (a.hi + keys - 1) / keys);
    a.cost = a.steps ? a.steps + p.extra : 0;
    return a;
}

template <bool kSome>
__device__ __forceinline__ AttendUnit attend_unit(const AttendParams &p, int u) {
    return attend_unit<kSome>(p, u, attend_raw(p, u));
}

// The unit behind u; blocks behind a sequence's last row are passed over.
__device__ __forceinline__ int attend_next(const AttendParams &p, const AttendUnit &a, int u) {
    return a.steps == 0 || a.row0 + a.rows >= a.n * p.group ? (a.list + 1) * p.blocks : u + 1;
}

// The first unit behind sequence b that somebody has to work on, or n_units: 32
// sequences are looked at together, so that a batch whose places are mostly empty
// is not walked one latency after the other.  The whole warp asks for one b.
template <bool kSome>
__device__ __noinline__ int attend_next_seq(const AttendParams &p, int b) {
    const int lists = p.n_kv_heads * p.blocks;
    for (++b; b < p.n_seqs; b += 32) {
        const int i = b + (threadIdx.x & 31);
        const unsigned has = __ballot_sync(0xffffffffu, i < p.n_seqs && attend_unit<kSome>(p, i * lists).steps > 0);
        if (has) return (b + __ffs(has) - 1) * lists;
    }
    return p.n_units;
}

// Cached rows that row r of the unit sees.
__device__ __forceinline__ int attend_sees(const AttendParams &p, const AttendUnit &a, int r) {
    return max(0, a.len - a.n + p.by_group(a.row0 + r) + 1);
}
// Its row of out [n_tokens][n_q_heads].
__device__ __forceinline__ int64_t attend_out_row(const AttendParams &p, const AttendUnit &a, int r) {
    const int token = p.by_group(a.row0 + r);
    return (int64_t)(a.q0 + token) * p.n_q_heads + a.h * p.group + (a.row0 + r - token * p.group);
}

// A page number that may be used: the pool's, or -1 (rows of zeros).
__device__ __forceinline__ int attend_page(const AttendParams &p, int list, int j) {
    const int page = p.table[(int64_t)list * p.max_pages + j];
    if (page < 0 || page >= p.n_pages) {
        set_status(p.status, KVC_DEV_BAD_PAGE);
        return -1;
    }
    return page;
}

// The CTA's run and the unit it begins in.
struct AttendRun {
    int64_t total, lo, hi;   // cost of all; this CTA's part
    int grid;                // CTAs with work
    int unit;                // first unit ...
    int64_t unit_lo;         // ... where that begins
    AttendRaw raw;           // ... and what it is made of
};

// (Where the products fit 32 bits the divisions are of 32 bits: a third of the
// instructions.)
__device__ __forceinline__ int64_t attend_cut(int64_t total, int grid, int c) {
    if (total * grid <= UINT_MAX) return (uint32_t)total * (uint32_t)c / (uint32_t)grid;
    return total * c / grid;
}
// The CTA whose run holds x.
__device__ __forceinline__ int attend_cta_of(int64_t total, int grid, int64_t x) {
    if (total * grid <= UINT_MAX) return (int)(((uint32_t)(x + 1) * (uint32_t)grid - 1) / (uint32_t)total);
    return (int)(((x + 1) * grid - 1) / total);
}

// The sum over a warp, in every lane.
__device__ __forceinline__ int64_t attend_warp_sum(int64_t x) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
// The sum over a warp's lanes up to this one.
__device__ __forceinline__ int64_t attend_warp_scan(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}
__device__ __forceinline__ AttendRaw attend_raw_of(const AttendRaw &raw, int lane) {
    return AttendRaw{__shfl_sync(0xffffffffu, raw.q0, lane), __shfl_sync(0xffffffffu, raw.q1, lane),
                     __shfl_sync(0xffffffffu, raw.len, lane)};
}

// The cost of the lane's list (0 where !real); a list of several units is added
// up by the whole warp.
template <bool kSome>
__device__ __forceinline__ int64_t attend_list_cost(const AttendParams &p, int list, bool real, AttendRaw *raw) {
    const int lane = threadIdx.x & 31;
    *raw = attend_raw(p, real ? list * p.blocks : p.n_units);
    int64_t cost = 0;
    int rows = 0;
    if (real) {
        const AttendUnit a = attend_unit<kSome>(p, list * p.blocks, *raw);
        cost = a.cost;
        rows = a.n * p.group;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, rows > p.unit_rows); left; left &= left - 1) {
        const int of = __ffs(left) - 1, u0 = __shfl_sync(0xffffffffu, list, of) * p.blocks;
        const int all = __shfl_sync(0xffffffffu, rows, of);
        const AttendRaw r = attend_raw_of(*raw, of);
        int64_t sum = 0;
        for (int i = lane; i < p.blocks && (int64_t)i * p.unit_rows < all; i += 32)
            sum += attend_unit<kSome>(p, u0 + i, r).cost;
        sum = attend_warp_sum(sum);
        if (lane == of) cost = sum;
    }
    return cost;
}

// The run without its unit.
__device__ __forceinline__ bool attend_run(int64_t total, AttendRun *r) {
    r->total = total;
    r->grid = (int)min((int64_t)gridDim.x, total);
    const bool works = (int)blockIdx.x < r->grid;
    r->lo = works ? attend_cut(total, r->grid, blockIdx.x) : 0;
    r->hi = works ? attend_cut(total, r->grid, blockIdx.x + 1) : 0;
    return works;
}

// The plan by lists: each warp adds up a stretch of them; the one whose stretch the
// CTA's run begins in looks for the unit, 32 lists and then 32 units at a time.  The total.
template <int NT, bool kSome>
__device__ __noinline__ int64_t attend_plan_lists(const AttendParams &p, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lists = p.n_seqs * p.n_kv_heads, per = (lists + NT / 32 - 1) / (NT / 32);
    const int l0 = min(lists, warp * per), l1 = min(lists, l0 + per);
    AttendRaw raw;
    int64_t mine = 0;
    for (int l = l0; l < l1; l += 32) mine += attend_list_cost<kSome>(p, l + lane, l + lane < l1, &raw);
    mine = attend_warp_sum(mine);
    if (lane == 0) scratch[warp] = mine;
    __syncthreads();
    int64_t at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) at += scratch[w];
        total += scratch[w];
    }
    int64_t *found = scratch + NT / 32;
    AttendRun r;
    const bool works = attend_run(total, &r);
    if (works && r.lo >= at && r.lo < at + mine) {
        for (int l = l0; l < l1; l += 32) {
            const int64_t cost = attend_list_cost<kSome>(p, l + lane, l + lane < l1, &raw);
            const int64_t end = at + attend_warp_scan(cost);
            const unsigned past = __ballot_sync(0xffffffffu, r.lo < end);
            if (past == 0) {
                at = __shfl_sync(0xffffffffu, end, 31);
                continue;
            }
            const int of = __ffs(past) - 1;
            at = __shfl_sync(0xffffffffu, end - cost, of);
            raw = attend_raw_of(raw, of);
            for (int i = 0; i < p.blocks; i += 32) {
                const int u = (l + of) * p.blocks + i + lane;
                const int64_t c = i + lane < p.blocks ? attend_unit<kSome>(p, u, raw).cost : 0;
                const int64_t until = at + attend_warp_scan(c);
                const unsigned beyond = __ballot_sync(0xffffffffu, r.lo < until);
                if (beyond == 0) {
                    at = __shfl_sync(0xffffffffu, until, 31);
                    continue;
                }
                if (lane == __ffs(beyond) - 1) {
                    found[0] = u;
                    found[1] = until - c;
                    found[2] = (int64_t)((uint64_t)(uint32_t)raw.q0 << 32 | (uint32_t)raw.q1);
                    found[3] = raw.len;
                }
                break;
            }
            break;
        }
    }
    return total;
}

// Every thread of a block of NT threads calls it; scratch: NT / 32 + 4 int64.
// By units: each thread adds up a stretch of them.  Where lists of several units
// make more than four per thread, by lists: a chunk's units would be one thread's
// (2,048 tokens and 255 decoding sequences, 64K units of which 2,300 have work:
// 362 us by units, 294 by lists, in one bf16 term; with one unit a list or few units the plan by
// lists takes 1 us longer).
template <int NT, bool kSome>
__device__ AttendRun attend_plan(const AttendParams &p, int64_t *scratch) {
    int64_t *found = scratch + NT / 32;
    AttendRun r;
    bool works;
    if (p.blocks > 1 && p.n_units > 4 * NT) {
        works = attend_run(attend_plan_lists<NT, kSome>(p, scratch), &r);
    } else {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = p.n_units / NT + 1;
        const int u0 = (int)min((int64_t)p.n_units, (int64_t)per * threadIdx.x), u1 = min(p.n_units - u0, per) + u0;
        int64_t mine = 0;
        for (int u = u0; u < u1;) {
            const AttendUnit a = attend_unit<kSome>(p, u);
            mine += a.cost;
            u = attend_next(p, a, u);
        }
        const int64_t x = attend_warp_scan(mine);
        if (lane == 31) scratch[warp] = x;
        __syncthreads();
        int64_t before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += scratch[w];
            total += scratch[w];
        }
        works = attend_run(total, &r);
        int64_t at = before + x - mine;
        if (works && r.lo >= at && r.lo < at + mine) {
            for (int u = u0; u < u1;) {
                const AttendRaw raw = attend_raw(p, u);
                const AttendUnit a = attend_unit<kSome>(p, u, raw);
                if (r.lo < at + a.cost) {
                    found[0] = u;
                    found[1] = at;
                    found[2] = (int64_t)((uint64_t)(uint32_t)raw.q0 << 32 | (uint32_t)raw.q1);
                    found[3] = raw.len;
                    break;
                }
                at += a.cost;
                u = attend_next(p, a, u);
            }
        }
    }
    __syncthreads();
    r.unit = works ? (int)found[0] : 0;
    r.unit_lo = works ? found[1] : 0;
    r.raw = works ? AttendRaw{(int)(found[2] >> 32), (int)(uint32_t)found[2], (int)found[3]} : AttendRaw{0, 0, 0};
    return r;
}

// ln of the row's sum = ln 2 (m + log2 l).
__device__ __forceinline__ void attend_store_lse(const AttendParams &p, int64_t row, float m, float l,
                                                 bool sees) {
    if (p.lse) p.lse[row] = sees ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

// A warp's rows of a slot are written: count it.  True, in the whole warp, if it
// is the last of `all`; then every other's rows are visible to it.  The counter
// is back at zero after that.  One alone is not counted: a group of one CTA,
// its unit's last, shares its counter with the group that the next unit may begin
// in that CTA, and the others of that one may have counted already.
__device__ __forceinline__ bool attend_last(uint32_t *count, uint32_t all) {
    __syncwarp();
    if (all == 1) return true;
    uint32_t before = 0;
    if ((threadIdx.x & 31) == 0) {
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
        if (before == all - 1) *count = 0;
    }
    before = __shfl_sync(0xffffffffu, before, 0);
    __syncwarp();   // lane 0's acquire is the warp's: a shuffle alone orders no memory
    return before == all - 1;
}

// How many warps have been counted; what they wrote before is visible after it.
__device__ __forceinline__ uint32_t attend_peek(const uint32_t *count) {
    uint32_t is = 0;
    if ((threadIdx.x & 31) == 0)
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(is) : "l"(count) : "memory");
    is = __shfl_sync(0xffffffffu, is, 0);
    __syncwarp();   // as in attend_last
    return is;
}

// Slots of a CTA: its first unit's (begun by an earlier CTA), its last unit's.
constexpr int kSlotFirst = 0, kSlotLast = 1;

__device__ __forceinline__ void attend_store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void attend_store4(__nv_bfloat16 *p, float4 x) {
    uint32_t a, b;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(x.w), "f"(x.z));
    *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}

// Joining: a unit shared by few CTAs is joined by the one that finishes last.  Of
// many, every kJoinGroup neighbours' slots are joined first, into the first
// one's, by the last of those: one SM reading 150 slots would take longer than
// all SMs took for their steps.
constexpr int kJoinAtOnce = 24, kJoinGroup = 12;
__device__ __forceinline__ int attend_groups(int ctas) {
    return ctas <= kJoinAtOnce ? 1 : (ctas + kJoinGroup - 1) / kJoinGroup;
}

struct AttendSpan {
    int c0;         // the unit's first CTA
    int from, step, n;   // slots of CTAs from, from + step, ..
    bool groups;    // they are joined groups
    bool out;       // the result is the output, else a group's
};

// Rows first.. of the unit; their places in the slots begin at slot_row.  `me`
// of `threads` threads; U chunks of four columns times S slots are asked for at a
// time.
template <typename T, int U, int S>
__device__ __noinline__ void attend_join(const AttendParams &p, const AttendUnit &a, const AttendSpan &s,
                                         int first, int rows, int slot_row, int me, int threads) {
    const int D = p.dim, quads = D / 4;
    // slot k of the span is slot0 + k * stride - (k > 0 and it begins with the
    // unit's first CTA): one 64-bit offset per slot, one addition per load
    const bool whole = s.from == s.c0;
    const int64_t slot0 = (int64_t)s.from * p.slots + (whole ? kSlotLast : kSlotFirst);
    const int64_t stride = (int64_t)s.step * p.slots, back = whole ? kSlotLast - kSlotFirst : 0;
    const int64_t slot_floats = (int64_t)p.slot_rows * D;
    const float2 *stat = (s.groups ? p.group_stat : p.stat) + slot_row;
    float *part = p.part + (int64_t)slot_row * D;
    for (int x0 = me; x0 < rows * quads; x0 += threads * U) {
        float top[U], sum[U];
        float4 acc[U];
        const float2 *stat_at[U];
        const float *part_at[U];
        bool real[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * threads, row = p.by_quads(x), col = (x - row * quads) * 4;
            real[u] = row < rows;
            stat_at[u] = stat + (real[u] ? row : 0);
            part_at[u] = part + (real[u] ? row * D + col : 0);
            top[u] = -INFINITY;
            sum[u] = 0.f;
            acc[u] = make_float4(0, 0, 0, 0);
        }
        for (int k0 = 0; k0 < s.n; k0 += S) {
            float2 st[U][S];
            float4 y[U][S];
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const bool is = k0 + k < s.n;
                const int64_t slot = slot0 + (is ? (k0 + k) * stride - (k0 + k > 0 ? back : 0) : 0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    st[u][k] = __ldcg(stat_at[u] + slot * p.slot_rows);
                    y[u][k] = __ldcg(reinterpret_cast<const float4 *>(part_at[u] + slot * slot_floats));
                }
                if (!is) {   // the span's first slot once more, with no weight
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        st[u][k] = make_float2(-INFINITY, 0.f);
                        y[u][k] = make_float4(0, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float t = top[u];
#pragma unroll
                for (int k = 0; k < S; ++k) t = fmaxf(t, st[u][k].x);
                const float ref = t == -INFINITY ? 0.f : t, down = ex2(top[u] - ref);
                top[u] = t;
                sum[u] *= down;
                acc[u] = make_float4(acc[u].x * down, acc[u].y * down, acc[u].z * down, acc[u].w * down);
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    const float w = ex2(st[u][k].x - ref);
                    sum[u] = fmaf(st[u][k].y, w, sum[u]);
                    acc[u].x = fmaf(y[u][k].x, w, acc[u].x);
                    acc[u].y = fmaf(y[u][k].y, w, acc[u].y);
                    acc[u].z = fmaf(y[u][k].z, w, acc[u].z);
                    acc[u].w = fmaf(y[u][k].w, w, acc[u].w);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!real[u]) continue;
            const int x = x0 + u * threads, row = p.by_quads(x), col = (x - row * quads) * 4;
            if (!s.out) {   // this thread alone has read this chunk of the slot
                *reinterpret_cast<float4 *>(part + slot0 * slot_floats + row * D + col) = acc[u];
                if (col == 0) p.group_stat[slot0 * p.slot_rows + slot_row + row] = make_float2(top[u], sum[u]);
                continue;
            }
            const bool see = attend_sees(p, a, first + row) > 0;
            const int64_t out_row = attend_out_row(p, a, first + row);
            const float inv = 1.f / sum[u];
            const float4 r = see ? make_float4(acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv)
                                 : make_float4(0, 0, 0, 0);
            attend_store4(static_cast<T *>(p.out) + out_row * D + col, r);
            if (col == 0) attend_store_lse(p, out_row, top[u], sum[u], see);
        }
    }
}


// What a launch needs of the workspace.
struct AttendNeeds {
    int grid, slots, slot_rows;
};
AttendNeeds attend_simt_needs(int sms);
AttendNeeds attend_tc_needs(int sms);
bool attend_tc_takes(int dtype, int dim, int group);
// The units' shape: blocks of unit_rows rows, of lists that have more than
// rows_above and at most rows_upto.  False if there are too many.
inline bool attend_units(AttendParams &p, int unit_rows, int rows_above, int rows_upto) {
    p.unit_rows = unit_rows;
    p.rows_above = rows_above;
    p.rows_upto = rows_upto;
    p.blocks = (std::min(p.max_new * p.group, rows_upto) + unit_rows - 1) / unit_rows;
    const int64_t n = (int64_t)p.n_seqs * p.n_kv_heads * p.blocks;
    p.n_units = (int)n;
    p.by_group = Divider((uint32_t)p.group);
    p.by_heads = Divider((uint32_t)p.n_kv_heads);
    p.by_blocks = Divider((uint32_t)p.blocks);
    p.by_quads = Divider((uint32_t)p.dim / 4);
    return n < INT_MAX;
}
// Both set the units' shape.
int launch_attend_simt(AttendParams &p, bool f32, int grid, cudaStream_t st);
int launch_attend_tc(AttendParams &p, int grid, cudaStream_t st);

}  // namespace kvc
