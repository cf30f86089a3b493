// pages_quant.cu -- rows of a paged cache held in 4 or 8 bits (quant.cuh): written,
// moved and read back.
//
// Lists, tables and pages are pages.cu's, and so is the plan of a call that takes
// pages; only what a row is made of differs.  Four lanes work out a group together,
// eight channels each: minimum and maximum by two shuffles, then every lane its own
// codes.  K and V of a row are the same lanes' work.
//
// What bounds them, measured on one GB300 with 560,000 rows of 128 in bf16 and 4 bits
// (368 MB there and as many back: 54 us each at the measured copy rate): writing takes 106
// us and 71% of the issue slots (the range, the step and the rounding, 170 instructions
// per eight channels of K and V in a warp); reading back 77 us, 4.8 TB/s, waiting for the
// rows.  In 8 bits 140,000 rows come back in 27 us, 5.4 TB/s.
#include "pages.cuh"
#include "quant.cuh"

namespace kvc {

namespace {

// Eight channels as they come, and as floats.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        if (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint4 b = v[sizeof(T) / 2 - 1];
            const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __uint_as_float(w[i]);
                x[4 + i] = __uint_as_float(y[i]);
            }
        }
    }
};
// Eight channels that come as bf16 pairs.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const uint32_t (&y)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store8(float *p, const uint32_t (&y)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        reinterpret_cast<float4 *>(p)[i] = make_float4(__uint_as_float(y[2 * i] << 16), __uint_as_float(y[2 * i] & 0xffff0000u),
                                                       __uint_as_float(y[2 * i + 1] << 16), __uint_as_float(y[2 * i + 1] & 0xffff0000u));
}

constexpr int kAtOnce = 4;   // parts that a lane reads before it goes on with the first

// A warp's rows are looked up 32 at a time, a lane each, and worked on in parts, 32 of
// any rows at a time: the search for a row's list and pages would cost as much as a
// part's work (560,000 rows of 128 read back from 4 bits: 116 us with a search per part,
// 102 so, 77 with four parts' loads in flight).
// Eight blocks per SM are launched, of which three to five are resident: the later ones
// fill what the earlier leave.  As many as are resident took 82 us instead of 77 to read
// and 113 instead of 106 to append those rows; twice as many, 78 and 109.  Moving rows is
// one round per warp either way, and gains from fewer (243,000 rows: 23 us, 19 so).
constexpr int kCompactPerSm = 5;

__device__ __forceinline__ int64_t of_lane(int64_t x, int lane) {
    return (int64_t)((uint64_t)__shfl_sync(0xffffffffu, (uint32_t)((uint64_t)x >> 32), lane) << 32 | __shfl_sync(0xffffffffu, (uint32_t)x, lane));
}

template <typename T>
struct AppendParams : MoveLists {
    int dim, groups;
    Divider by_pieces;        // pieces of eight channels of a row, 4 * groups
    const T *k_src, *v_src;
    uint8_t *k_pool, *v_pool;
};

template <int BITS, typename T>
__global__ void __launch_bounds__(kMoveThreads) append_quant_kernel(const __grid_constant__ AppendParams<T> p) {
    let_next_start();
    wait_for_inputs();
    if (!p.s.head->ok) return;
    const int64_t rows = p.s.head->total_rows;
    const int lane = threadIdx.x & 31, pieces = 4 * p.groups;
    const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
    const int64_t me = ((int64_t)blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    enter_pages(p, me, warps);
    const int64_t per = (rows + warps - 1) / warps;
    const int64_t r0 = me * per, r1 = min(rows, r0 + per);
    if (r0 >= r1) return;
    int i = owner(p.s.row_begin, p.n_lists, r0);
    uint32_t bad = 0;
    for (int64_t at = r0; at < r1; at += 32) {
        MovedRow m{0, 0, false};
        if (at + lane < r1) {
            i = owner_from(p.s.row_begin, p.n_lists, at + lane, i);
            m = moved_row<true>(p, i, at + lane, &bad);
        }
        // in a copied row `from` counts the pool's rows, and is negative here
        const int64_t from_of = m.own_pool ? -1 - m.from : m.from;
        const int items = (int)min((int64_t)32, r1 - at) * pieces;   // a multiple of four: groups' lanes stay together
        // the lane's part number base / 32: its source (negative: copied) and values
        Eight<T> k_next, v_next;
        int64_t from_next = 0;
        int u_next = 0, dr_next = 0;
        auto look = [&](int base) {
            const int it = base + lane, dr = p.by_pieces(it);
            u_next = it - dr * pieces;
            dr_next = dr & 31;
            from_next = of_lane(from_of, dr_next);
            k_next.clear();
            v_next.clear();
            if (it < items && from_next >= 0 && u_next * 8 < p.dim) {
                k_next.load(p.k_src + from_next * p.dim + u_next * 8);
                v_next.load(p.v_src + from_next * p.dim + u_next * 8);
            }
        };
        look(0);
        for (int base = 0; base < items; base += 32) {
            const int64_t from = from_next, to_row = of_lane(m.to, dr_next);
            const int g = u_next >> 2, c = u_next & 3;
            float kx[8], vx[8];
            k_next.floats(kx);
            v_next.floats(vx);
            look(base + 32);
            const unsigned together = __ballot_sync(0xffffffffu, base + lane < items);
            if (base + lane >= items) continue;
            const QuantRow to = quant_row(BITS, p.groups, to_row);
            if (from < 0) {   // a shared last page's row, as it is (whole groups of lanes are, or none)
                const QuantRow held = quant_row(BITS, p.groups, -1 - from);
                quant_store<BITS>(p.k_pool + to.codes, p.groups, g, c, false, quant_load<BITS>(p.k_pool + held.codes, p.groups, g, c, false));
                quant_store<BITS>(p.v_pool + to.codes, p.groups, g, c, true, quant_load<BITS>(p.v_pool + held.codes, p.groups, g, c, true));
                if (c == 0) {
                    reinterpret_cast<uint16_t *>(p.k_pool + to.words)[g] = reinterpret_cast<const uint16_t *>(p.k_pool + held.words)[g];
                    reinterpret_cast<uint16_t *>(p.v_pool + to.words)[g] = reinterpret_cast<const uint16_t *>(p.v_pool + held.words)[g];
                }
                continue;
            }
            uint32_t kw, vw;
            uint2 kc, vc;
            quant_encode<BITS>(kx, vx, together & 0xfu << (lane & 28), &kc, &kw, &vc, &vw);
            quant_store<BITS>(p.k_pool + to.codes, p.groups, g, c, false, kc);
            quant_store<BITS>(p.v_pool + to.codes, p.groups, g, c, true, vc);
            if (c == 0) {
                reinterpret_cast<uint16_t *>(p.k_pool + to.words)[g] = (uint16_t)kw;
                reinterpret_cast<uint16_t *>(p.v_pool + to.words)[g] = (uint16_t)vw;
            }
        }
        __syncwarp();
    }
}

struct CompactParams : MoveLists {
    int groups;
    Divider by_groups;
    uint8_t *k_pool, *v_pool;
};

// Rows as they are: a lane moves 16 (4 bits) or 32 bytes of codes of K and of V,
// and the words of one group.
template <int BITS>
__global__ void __launch_bounds__(kMoveThreads, kCompactPerSm) compact_quant_kernel(const __grid_constant__ CompactParams p) {
    let_next_start();
    wait_for_inputs();
    if (!p.s.head->ok) return;
    const int64_t rows = p.s.head->total_rows;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
    const int64_t me = ((int64_t)blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    const int64_t per = (rows + warps - 1) / warps;
    const int64_t r0 = me * per, r1 = min(rows, r0 + per);
    if (r0 >= r1) return;
    int i = owner(p.s.row_begin, p.n_lists, r0);
    uint32_t bad = 0;
    constexpr int kVecs = BITS / 4;
    for (int64_t at = r0; at < r1; at += 32) {
        MovedRow m{-1, 0, true};
        if (at + lane < r1) {
            i = owner_from(p.s.row_begin, p.n_lists, at + lane, i);
            m = moved_row<false>(p, i, at + lane, &bad);
        }
        const int items = (int)min((int64_t)32, r1 - at) * p.groups;
        for (int base = 0; base < items; base += 32) {
            const int it = base + lane, dr = p.by_groups(it), g = it - dr * p.groups;
            const int64_t from_row = of_lane(m.from, dr & 31), to_row = of_lane(m.to, dr & 31);
            if (it >= items) continue;
            uint4 k[kVecs] = {}, v[kVecs] = {};   // a row of zeros has steps of zero
            uint16_t kw = 0, vw = 0;
            if (from_row >= 0) {
                const QuantRow from = quant_row(BITS, p.groups, from_row);
#pragma unroll
                for (int e = 0; e < kVecs; ++e) {
                    k[e] = reinterpret_cast<const uint4 *>(p.k_pool + from.codes)[g * kVecs + e];
                    v[e] = reinterpret_cast<const uint4 *>(p.v_pool + from.codes)[g * kVecs + e];
                }
                kw = reinterpret_cast<const uint16_t *>(p.k_pool + from.words)[g];
                vw = reinterpret_cast<const uint16_t *>(p.v_pool + from.words)[g];
            }
            const QuantRow to = quant_row(BITS, p.groups, to_row);
#pragma unroll
            for (int e = 0; e < kVecs; ++e) {
                reinterpret_cast<uint4 *>(p.k_pool + to.codes)[g * kVecs + e] = k[e];
                reinterpret_cast<uint4 *>(p.v_pool + to.codes)[g * kVecs + e] = v[e];
            }
            reinterpret_cast<uint16_t *>(p.k_pool + to.words)[g] = kw;
            reinterpret_cast<uint16_t *>(p.v_pool + to.words)[g] = vw;
        }
        __syncwarp();
    }
    if (bad) set_status(&p.s.head->status, bad);
}

struct ReadPlan {
    PagesState s;
    const int32_t *len, *first, *counts;
    const int64_t *dst_row;
    int64_t dst_step, dst_rows;
    int32_t n_lists, max_pages, shift;
};

// Rows of every list, added up; nothing is read unless all of it is in range.
__global__ void __launch_bounds__(kPlanThreads) read_plan_kernel(ReadPlan p) {
    __shared__ Two scratch[33];
    __shared__ uint32_t s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    let_next_start();
    wait_for_inputs();
    __syncthreads();
    const int64_t most = (int64_t)p.max_pages << p.shift;
    bool bad = false;
    int64_t sum = 0;
    for (int base = 0; base < p.n_lists; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        Two need{0, 0}, all;
        if (i < p.n_lists && p.counts[i] > 0) {
            const int64_t n = p.counts[i], from = p.first ? p.first[i] : 0, len = p.len[i], to = p.dst_row[i];
            need.rows = n;
            bad |= len < 0 || len > most || from < 0 || from + n > len || to < 0 || to >= p.dst_rows ||
                   (n > 1 && p.dst_step > 0 && n - 1 > (p.dst_rows - 1 - to) / p.dst_step);
        }
        const Two at = block_scan(need, scratch, &all);
        if (i < p.n_lists) p.s.row_begin[i] = sum + at.rows;
        sum += all.rows;
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) {
        if (s_bad) set_status(&p.s.head->status, KVC_DEV_BAD_LIST);
        p.s.head->ok = !s_bad;
        p.s.head->total_rows = sum;
    }
}

template <typename T>
struct ReadParams {
    PagesState s;
    const int32_t *table, *first;
    const int64_t *dst_row;
    int64_t dst_step;
    int32_t n_lists, n_pages, max_pages, shift, dim, groups;
    Divider by_pieces;        // pieces of eight channels of a row, dim / 8
    const uint8_t *k_pool, *v_pool;
    T *k_dst, *v_dst;
};

template <int BITS, typename T>
__global__ void __launch_bounds__(kMoveThreads) read_quant_kernel(const __grid_constant__ ReadParams<T> p) {
    let_next_start();
    wait_for_inputs();
    if (!p.s.head->ok) return;
    const int64_t rows = p.s.head->total_rows;
    const int lane = threadIdx.x & 31, ps = 1 << p.shift, pieces = p.dim / 8;
    const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
    const int64_t me = ((int64_t)blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    const int64_t per = (rows + warps - 1) / warps;
    const int64_t r0 = me * per, r1 = min(rows, r0 + per);
    if (r0 >= r1) return;
    int i = owner(p.s.row_begin, p.n_lists, r0);
    bool bad = false;
    for (int64_t at = r0; at < r1; at += 32) {
        int64_t from_of = -1, to_of = 0;   // row of the pools, -1: zeros; element of the destination
        if (at + lane < r1) {
            const int64_t r = at + lane;
            i = owner_from(p.s.row_begin, p.n_lists, r, i);
            const int64_t k = r - p.s.row_begin[i];
            const int row = (p.first ? p.first[i] : 0) + (int)k;
            const int page = p.table[(int64_t)i * p.max_pages + (row >> p.shift)];
            to_of = (p.dst_row[i] + k * p.dst_step) * p.dim;
            if (page >= 0 && page < p.n_pages)
                from_of = ((int64_t)page << p.shift) + (row & (ps - 1));
            else
                bad = true;
        }
        const int items = (int)min((int64_t)32, r1 - at) * pieces;
        for (int base = 0; base < items; base += 32 * kAtOnce) {
            uint2 kc[kAtOnce], vc[kAtOnce];
            uint32_t kw[kAtOnce], vw[kAtOnce];
            int64_t to[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int it = base + 32 * e + lane, dr = p.by_pieces(it), u = it - dr * pieces;
                const int64_t from = of_lane(from_of, dr & 31);
                to[e] = of_lane(to_of, dr & 31) + u * 8;
                if (it >= items) to[e] = -1;
                kc[e] = vc[e] = make_uint2(0, 0);
                kw[e] = vw[e] = 0;   // rows of zeros
                if (it < items && from >= 0) {
                    const QuantRow held = quant_row(BITS, p.groups, from);
                    const int g = u >> 2, c = u & 3;
                    if (p.k_dst) {
                        kc[e] = quant_load<BITS>(p.k_pool + held.codes, p.groups, g, c, false);
                        kw[e] = reinterpret_cast<const uint16_t *>(p.k_pool + held.words)[g];
                    }
                    if (p.v_dst) {
                        vc[e] = quant_load<BITS>(p.v_pool + held.codes, p.groups, g, c, true);
                        vw[e] = reinterpret_cast<const uint16_t *>(p.v_pool + held.words)[g];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                if (to[e] < 0) continue;
                uint32_t y[4];
                if (p.k_dst) {
                    quant_bf16<BITS>(kc[e], kw[e] * 0x10001u, y);
                    store8(p.k_dst + to[e], y);
                }
                if (p.v_dst) {
                    quant_bf16<BITS>(vc[e], vw[e] * 0x10001u, y);
                    store8(p.v_dst + to[e], y);
                }
            }
        }
        __syncwarp();
    }
    if (bad) set_status(&p.s.head->status, KVC_DEV_BAD_PAGE);
}

template <int BITS, typename T>
void launch_append(const MoveLists &m, int dim, const void *k_src, const void *v_src, void *k_pool, void *v_pool,
                   int sms, cudaStream_t st) {
    const int groups = quant_groups(dim);
    const AppendParams<T> p{m, dim, groups, Divider(4 * groups), static_cast<const T *>(k_src),
                            static_cast<const T *>(v_src), static_cast<uint8_t *>(k_pool),
                            static_cast<uint8_t *>(v_pool)};
    launch_early(append_quant_kernel<BITS, T>, sms * 8, kMoveThreads, 0, st, p);
}

template <int BITS, typename T>
void launch_read(ReadParams<T> p, const void *k_pool, const void *v_pool, void *k_dst, void *v_dst, int sms,
                 cudaStream_t st) {
    p.k_pool = static_cast<const uint8_t *>(k_pool);
    p.v_pool = static_cast<const uint8_t *>(v_pool);
    p.k_dst = static_cast<T *>(k_dst);
    p.v_dst = static_cast<T *>(v_dst);
    launch_early(read_quant_kernel<BITS, T>, sms * 8, kMoveThreads, 0, st, p);
}

}  // namespace

int launch_pages_append_quant(const kvc_cache &c, int bits, const PagesState &s, int32_t *table, int32_t *len,
                              int32_t n_lists, const int32_t *counts, const int64_t *src_row, int64_t src_step,
                              const void *k_src, const void *v_src, int64_t src_rows, void *k_pool, void *v_pool,
                              int sms, cudaStream_t st) {
    const int shift = log2_of(c.page_rows);
    launch_pages_plan({s, table, len, counts, src_row, src_step, src_rows, n_lists, c.n_pages, c.max_pages, shift, 0,
                       true}, st);
    const MoveLists m{s, table, src_row, src_step, nullptr, n_lists, c.n_pages, c.max_pages, shift, 0};
    const bool f32 = c.dtype == KVC_F32;
    if (bits == 4)
        f32 ? launch_append<4, float>(m, c.head_dim, k_src, v_src, k_pool, v_pool, sms, st)
            : launch_append<4, __nv_bfloat16>(m, c.head_dim, k_src, v_src, k_pool, v_pool, sms, st);
    else
        f32 ? launch_append<8, float>(m, c.head_dim, k_src, v_src, k_pool, v_pool, sms, st)
            : launch_append<8, __nv_bfloat16>(m, c.head_dim, k_src, v_src, k_pool, v_pool, sms, st);
    return cache_launched("kvc_pages_append_quant");
}

int launch_pages_compact_quant(const kvc_cache &c, int bits, const PagesState &s, int32_t *table, int32_t *len,
                               int32_t n_lists, const int32_t *idx, int32_t k_max, const int32_t *counts,
                               void *k_pool, void *v_pool, int sms, cudaStream_t st) {
    const int shift = log2_of(c.page_rows), groups = quant_groups(c.head_dim);
    launch_pages_plan({s, table, len, counts, nullptr, 0, 0, n_lists, c.n_pages, c.max_pages, shift, k_max, false}, st);
    const CompactParams p{{s, table, nullptr, 0, idx, n_lists, c.n_pages, c.max_pages, shift, k_max}, groups,
                          Divider(groups), static_cast<uint8_t *>(k_pool), static_cast<uint8_t *>(v_pool)};
    launch_early(bits == 4 ? compact_quant_kernel<4> : compact_quant_kernel<8>, sms * kCompactPerSm, kMoveThreads, 0, st, p);
    launch_pages_swap(c, s, table, len, n_lists, counts, st);
    return cache_launched("kvc_pages_compact_quant");
}

int launch_pages_read_quant(const kvc_cache &c, int bits, const PagesState &s, const int32_t *table,
                            const int32_t *len, int32_t n_lists, const int32_t *first, const int32_t *counts,
                            const int64_t *dst_row, int64_t dst_step, const void *k_pool, const void *v_pool,
                            void *k_dst, void *v_dst, int64_t dst_rows, int sms, cudaStream_t st) {
    const int shift = log2_of(c.page_rows), groups = quant_groups(c.head_dim);
    launch_early(read_plan_kernel, 1, kPlanThreads, 0, st,
                 ReadPlan{s, len, first, counts, dst_row, dst_step, dst_rows, n_lists, c.max_pages, shift});
    const Divider by(c.head_dim / 8);
    auto go = [&](auto type, auto of_bits) {
        using T = decltype(type);
        launch_read<decltype(of_bits)::value>(
            ReadParams<T>{s, table, first, dst_row, dst_step, n_lists, c.n_pages, c.max_pages, shift, c.head_dim, groups,
                          by, nullptr, nullptr, nullptr, nullptr},
            k_pool, v_pool, k_dst, v_dst, sms, st);
    };
    using Four = std::integral_constant<int, 4>;
    using Eight = std::integral_constant<int, 8>;
    if (c.dtype == KVC_F32)
        bits == 4 ? go(0.f, Four{}) : go(0.f, Eight{});
    else
        bits == 4 ? go(__nv_bfloat16{}, Four{}) : go(__nv_bfloat16{}, Eight{});
    return cache_launched("kvc_pages_read_quant");
}

}  // namespace kvc
