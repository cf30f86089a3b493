// attend_simt.cu -- attention of new tokens over the paged cache on the CUDA
// cores, fp32 throughout: fp32 caches, head sizes the tensor cores' kernel does
// not take, and groups of more than 128 query heads.
//
// One pass over the keys with a running maximum m and sum l per row (logits in
// log2 units, so that one ex2 gives a probability):
//   m' = max(m, max_j x_j),  l' = l 2^(m - m') + sum_j 2^(x_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(x_j - m') v_j,  out = o / l.
// A block holds kRows rows (tokens x query heads of one KV head) and walks 64-key
// tiles through shared memory; 16 x 16 threads each own kRows/16 rows x 4 keys of
// the logits and kRows/16 rows x D/16 columns of o.
#include "attend.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr int kSlotRows = 64;

template <int ROWS, int DMAX>
struct SimtSmem {
    float q[ROWS][DMAX + 4];
    float k[kKeys][DMAX + 4];
    float v[kKeys][DMAX];
    float pr[ROWS][kKeys + 4];
    int64_t plan[kThreads / 32 + 4];
    uint32_t last;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int ROWS, int DMAX>
__global__ void __launch_bounds__(kThreads) attend_simt_kernel(AttendParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    auto &s = *reinterpret_cast<SimtSmem<ROWS, DMAX> *>(raw);
    constexpr int RT = ROWS / 16, CT = DMAX / 16;   // rows and columns of a thread
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int D = p.dim, D4 = D / 4;
    const AttendRun run = attend_plan<kThreads>(p, s.plan);
    if (run.lo >= run.hi) return;
    int64_t u = run.unit, u_lo = run.unit_lo;
    for (int64_t pos = run.lo; pos < run.hi;) {
        const AttendUnit a = attend_unit(p, u);
        if (a.steps == 0) {
            u = attend_next(p, a, u);
            continue;
        }
        const int64_t end = min(run.hi, u_lo + a.steps);
        const int t0 = (int)(pos - u_lo), t1 = (int)(end - u_lo);
        const int rows = a.rows;
        __syncthreads();   // the unit before is done with q
        for (int i = tid; i < ROWS * D4; i += kThreads) {
            const int r = i / D4, c = (i - r * D4) * 4;
            float4 x = make_float4(0, 0, 0, 0);
            if (r < rows) {
                const int token = (a.row0 + r) / p.group, g = a.row0 + r - token * p.group;
                x = load4(static_cast<const T *>(p.q) + (a.q0 + token) * p.q_stride +
                          (int64_t)(a.h * p.group + g) * D + c);
            }
            *reinterpret_cast<float4 *>(&s.q[r][c]) = x;
        }
        float m[RT], l[RT], o[RT][CT];
        int sees[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty * RT + i;
            m[i] = -INFINITY;
            l[i] = 0.f;
            sees[i] = r < rows ? attend_sees(p, a, r) : 0;
#pragma unroll
            for (int c = 0; c < CT; ++c) o[i][c] = 0.f;
        }
        for (int t = t0; t < t1; ++t) {
            const int j0 = t * kKeys;
            __syncthreads();   // the tile before is done with k, v and pr
            for (int i = tid; i < kKeys * D4; i += kThreads) {
                const int j = i / D4, c = (i - j * D4) * 4;
                float4 kk = make_float4(0, 0, 0, 0), vv = kk;
                if (j0 + j < a.hi) {
                    const int page = attend_page(p, a.list, (j0 + j) >> p.shift);
                    if (page >= 0) {
                        const int64_t at = ((((int64_t)page << p.shift) + ((j0 + j) & ((1 << p.shift) - 1))) * D) + c;
                        kk = load4(static_cast<const T *>(p.k_pool) + at);
                        vv = load4(static_cast<const T *>(p.v_pool) + at);
                    }
                }
                *reinterpret_cast<float4 *>(&s.k[j][c]) = kk;
                *reinterpret_cast<float4 *>(&s.v[j][c]) = vv;
            }
            __syncthreads();
            // logits of rows ty*RT.. and keys tx, tx+16, tx+32, tx+48
            float x[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
            for (int c = 0; c < D; c += 4) {
                float4 kk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(&s.k[tx + 16 * j][c]);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&s.q[ty * RT + i][c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] = fmaf(qq.x, kk[j].x, x[i][j]);
                        x[i][j] = fmaf(qq.y, kk[j].y, x[i][j]);
                        x[i][j] = fmaf(qq.z, kk[j].z, x[i][j]);
                        x[i][j] = fmaf(qq.w, kk[j].w, x[i][j]);
                    }
                }
            }
            bool cut = false;   // some row of the thread sees only part of the tile
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int left = sees[i] - j0;
                cut |= left < kKeys;
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = tx + 16 * j < left ? x[i][j] * p.scale_log2 : -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                // all -inf so far: any finite reference gives 2^-inf = 0
                const float ref = top == -INFINITY ? 0.f : top;
                const float down = ex2(m[i] - ref);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = ex2(x[i][j] - ref);
                    sum += e;
                    s.pr[ty * RT + i][tx + 16 * j] = e;
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l[i] = l[i] * down + sum;
                m[i] = top;
#pragma unroll
                for (int c = 0; c < CT; ++c) o[i][c] *= down;
            }
            __syncthreads();
            const int nk = min(kKeys, a.hi - j0);
            for (int j = 0; j < nk; ++j) {
                float e[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) e[i] = s.pr[ty * RT + i][j];
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int col = tx + 16 * c;
                    if (col < D) {
                        const float vv = s.v[j][col];
                        if (!cut) {
#pragma unroll
                            for (int i = 0; i < RT; ++i) o[i][c] = fmaf(e[i], vv, o[i][c]);
                        } else {   // a value a row does not see may be anything
#pragma unroll
                            for (int i = 0; i < RT; ++i)
                                if (j0 + j < sees[i]) o[i][c] = fmaf(e[i], vv, o[i][c]);
                        }
                    }
                }
            }
        }
        // whole units go straight out, shared ones through the slots
        const bool whole = t0 == 0 && t1 == a.steps;
        const int slot = 2 * blockIdx.x + (t0 == 0 ? kSlotLast : kSlotFirst);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty * RT + i;
            if (r >= rows) continue;
            if (whole) {
                const int64_t row = attend_out_row(p, a, r);
                T *out = static_cast<T *>(p.out) + row * D;
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    if (tx + 16 * c < D) store1(out + tx + 16 * c, sees[i] > 0 ? o[i][c] / l[i] : 0.f);
                if (tx == 0) attend_store_lse(p, row, m[i], l[i], sees[i] > 0);
            } else {
                float *part = p.part + ((int64_t)slot * p.slot_rows + r) * D;
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    if (tx + 16 * c < D) part[tx + 16 * c] = o[i][c];
                if (tx == 0) p.stat[(int64_t)slot * p.slot_rows + r] = make_float2(m[i], l[i]);
            }
        }
        if (!whole) {
            const int c0 = attend_cta_of(run.total, run.grid, u_lo);
            const int c1 = attend_cta_of(run.total, run.grid, u_lo + a.steps - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t before = atomicAdd(&p.arrived[2 * c0], 1u);
                s.last = before == (uint32_t)(c1 - c0);
                if (s.last) p.arrived[2 * c0] = 0;
            }
            __syncthreads();
            if (s.last) {
                __threadfence();
                // thread = (row, 16 column lanes), as above
                for (int r = ty; r < rows; r += 16) {
                    float top = -INFINITY;
                    for (int c = c0; c <= c1; ++c)
                        top = fmaxf(top, __ldcg(&p.stat[(int64_t)(2 * c + (c == c0)) * p.slot_rows + r]).x);
                    const float ref = top == -INFINITY ? 0.f : top;
                    float sum = 0.f, acc[CT];
#pragma unroll
                    for (int i = 0; i < CT; ++i) acc[i] = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const int64_t at = (int64_t)(2 * c + (c == c0)) * p.slot_rows + r;
                        const float2 st = __ldcg(&p.stat[at]);
                        const float w = ex2(st.x - ref);
                        sum = fmaf(st.y, w, sum);
#pragma unroll
                        for (int i = 0; i < CT; ++i)
                            if (tx + 16 * i < D) acc[i] = fmaf(__ldcg(&p.part[at * D + tx + 16 * i]), w, acc[i]);
                    }
                    const bool any = attend_sees(p, a, r) > 0;
                    const int64_t row = attend_out_row(p, a, r);
                    T *out = static_cast<T *>(p.out) + row * D;
#pragma unroll
                    for (int i = 0; i < CT; ++i)
                        if (tx + 16 * i < D) store1(out + tx + 16 * i, any ? acc[i] / sum : 0.f);
                    if (tx == 0) attend_store_lse(p, row, top, sum, any);
                }
            }
        }
        pos = end;
        u_lo += a.steps;
        u = attend_next(p, a, u);
    }
}

template <typename T, int ROWS, int DMAX>
int launch(AttendParams &p, int grid, cudaStream_t st) {
    constexpr size_t bytes = sizeof(SimtSmem<ROWS, DMAX>);
    static_assert(bytes <= 232448, "shared memory of one block");
    cudaFuncSetAttribute(attend_simt_kernel<T, ROWS, DMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         (int)bytes);
    attend_simt_kernel<T, ROWS, DMAX><<<grid, kThreads, bytes, st>>>(p);
    return cache_launched("kvc_attend");
}

template <typename T>
int launch_rows(AttendParams &p, int rows, int grid, cudaStream_t st) {
    if (rows <= 16)
        return p.dim <= 64    ? launch<T, 16, 64>(p, grid, st)
               : p.dim <= 128 ? launch<T, 16, 128>(p, grid, st)
                              : launch<T, 16, 256>(p, grid, st);
    return p.dim <= 64    ? launch<T, 64, 64>(p, grid, st)
           : p.dim <= 128 ? launch<T, 64, 128>(p, grid, st)
                          : launch<T, 64, 256>(p, grid, st);
}

}  // namespace

AttendNeeds attend_simt_needs(int sms) { return {2 * sms, 2, kSlotRows}; }

int launch_attend_simt(AttendParams &p, bool f32, int grid, cudaStream_t st) {
    // 16 rows per block where a list's tokens fill no more
    const int rows = p.max_new * p.group <= 16 ? 16 : kSlotRows;
    p.unit_rows = rows;
    p.blocks = (p.max_new * p.group + rows - 1) / rows;
    p.n_units = (int64_t)p.n_seqs * p.n_kv_heads * p.blocks;
    p.step_keys = kKeys;
    p.split_rows = 0;
    return f32 ? launch_rows<float>(p, rows, grid, st) : launch_rows<__nv_bfloat16>(p, rows, grid, st);
}

}  // namespace kvc
