// pages_quant.cu -- rows of a paged cache held in 4 or 8 bits (quant.cuh): written,
// moved and read back.
//
// Lists, tables and pages are pages.cu's, and so is the plan of a call that takes
// pages; only what a row is made of differs.  Four lanes work out a group together,
// eight channels each: minimum and maximum by two shuffles, then every lane its own
// codes.  K and V of a row are the same lanes' work.
#include "pages.cuh"
#include "quant.cuh"

namespace kvc {

namespace {

// Eight channels as floats.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];   // exact: see quant.cuh
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a warp's next 32 items (parts of rows) begin: no 64-bit division per step.
struct Place {
    int64_t row;
    int item;
    __device__ __forceinline__ void next(const Divider &by) {
        const int rows = by(item += 32);
        row += rows;
        item -= rows * (int)by.d;
    }
};

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
    const int64_t items = (r1 - r0) * pieces;   // a multiple of four: groups' lanes stay together
    Place place{r0, 0};
    for (int64_t base = 0; base < items; base += 32, place.next(p.by_pieces)) {
        const int it = place.item + lane, dr = p.by_pieces(it), u = it - dr * pieces;
        const int64_t r = place.row + dr;
        const bool real = base + lane < items;
        const unsigned together = __ballot_sync(0xffffffffu, real);
        if (!real) break;
        i = owner_from(p.s.row_begin, p.n_lists, r, i);
        const MovedRow m = moved_row<true>(p, i, r, &bad);
        const int g = u >> 2, c = u & 3;
        const QuantRow to = quant_row(BITS, p.groups, m.to);
        uint2 kc, vc;
        uint32_t kw, vw;
        const bool copied = m.own_pool;
        if (copied) {   // a shared last page's row, as it is
            const QuantRow from = quant_row(BITS, p.groups, m.from);
            kc = quant_load<BITS>(p.k_pool + from.codes, p.groups, g, c, false);
            vc = quant_load<BITS>(p.v_pool + from.codes, p.groups, g, c, true);
            kw = reinterpret_cast<const uint16_t *>(p.k_pool + from.words)[g];
            vw = reinterpret_cast<const uint16_t *>(p.v_pool + from.words)[g];
        }
        float kx[8] = {}, vx[8] = {};
        if (!copied && u * 8 < p.dim) {
            load8(p.k_src + m.from * p.dim + u * 8, kx);
            load8(p.v_src + m.from * p.dim + u * 8, vx);
        }
        uint32_t kn, vn;
        const uint2 ke = quant_encode<BITS>(kx, together, &kn), ve = quant_encode<BITS>(vx, together, &vn);
        if (!copied) {
            kc = ke;
            vc = ve;
            kw = kn;
            vw = vn;
        }
        quant_store<BITS>(p.k_pool + to.codes, p.groups, g, c, false, kc);
        quant_store<BITS>(p.v_pool + to.codes, p.groups, g, c, true, vc);
        if (c == 0) {
            reinterpret_cast<uint16_t *>(p.k_pool + to.words)[g] = (uint16_t)kw;
            reinterpret_cast<uint16_t *>(p.v_pool + to.words)[g] = (uint16_t)vw;
        }
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
__global__ void __launch_bounds__(kMoveThreads) compact_quant_kernel(const __grid_constant__ CompactParams p) {
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
    const int64_t items = (r1 - r0) * p.groups;
    constexpr int kVecs = BITS / 4;
    Place place{r0, 0};
    for (int64_t base = 0; base + lane < items; base += 32, place.next(p.by_groups)) {
        const int it = place.item + lane, dr = p.by_groups(it), g = it - dr * p.groups;
        const int64_t r = place.row + dr;
        i = owner_from(p.s.row_begin, p.n_lists, r, i);
        const MovedRow m = moved_row<false>(p, i, r, &bad);
        uint4 k[kVecs] = {}, v[kVecs] = {};   // a row of zeros has steps of zero
        uint16_t kw = 0, vw = 0;
        if (m.from >= 0) {
            const QuantRow from = quant_row(BITS, p.groups, m.from);
#pragma unroll
            for (int e = 0; e < kVecs; ++e) {
                k[e] = reinterpret_cast<const uint4 *>(p.k_pool + from.codes)[g * kVecs + e];
                v[e] = reinterpret_cast<const uint4 *>(p.v_pool + from.codes)[g * kVecs + e];
            }
            kw = reinterpret_cast<const uint16_t *>(p.k_pool + from.words)[g];
            vw = reinterpret_cast<const uint16_t *>(p.v_pool + from.words)[g];
        }
        const QuantRow to = quant_row(BITS, p.groups, m.to);
#pragma unroll
        for (int e = 0; e < kVecs; ++e) {
            reinterpret_cast<uint4 *>(p.k_pool + to.codes)[g * kVecs + e] = k[e];
            reinterpret_cast<uint4 *>(p.v_pool + to.codes)[g * kVecs + e] = v[e];
        }
        reinterpret_cast<uint16_t *>(p.k_pool + to.words)[g] = kw;
        reinterpret_cast<uint16_t *>(p.v_pool + to.words)[g] = vw;
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
    const int64_t items = (r1 - r0) * pieces;
    Place place{r0, 0};
    for (int64_t base = 0; base + lane < items; base += 32, place.next(p.by_pieces)) {
        const int it = place.item + lane, dr = p.by_pieces(it), u = it - dr * pieces;
        const int64_t r = place.row + dr;
        i = owner_from(p.s.row_begin, p.n_lists, r, i);
        const int64_t at = r - p.s.row_begin[i];
        const int row = (p.first ? p.first[i] : 0) + (int)at;
        const int page = p.table[(int64_t)i * p.max_pages + (row >> p.shift)];
        const int64_t to = (p.dst_row[i] + at * p.dst_step) * p.dim + u * 8;
        float k[8] = {}, v[8] = {};
        if (page >= 0 && page < p.n_pages) {
            const QuantRow from = quant_row(BITS, p.groups, ((int64_t)page << p.shift) + (row & (ps - 1)));
            const int g = u >> 2, c = u & 3;
            if (p.k_dst)
                quant_values<BITS>(quant_load<BITS>(p.k_pool + from.codes, p.groups, g, c, false),
                                   reinterpret_cast<const uint16_t *>(p.k_pool + from.words)[g], k);
            if (p.v_dst)
                quant_values<BITS>(quant_load<BITS>(p.v_pool + from.codes, p.groups, g, c, true),
                                   reinterpret_cast<const uint16_t *>(p.v_pool + from.words)[g], v);
        } else {
            bad = true;
        }
        if (p.k_dst) store8(p.k_dst + to, k);
        if (p.v_dst) store8(p.v_dst + to, v);
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
    launch_early(bits == 4 ? compact_quant_kernel<4> : compact_quant_kernel<8>, sms * 8, kMoveThreads, 0, st, p);
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
