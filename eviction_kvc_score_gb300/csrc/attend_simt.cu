// attend_simt.cu -- attention of new tokens over the paged cache on the CUDA
// cores, fp32 throughout: fp32 caches, head sizes the tensor cores' kernel does
// not take, and groups of more than 128 query heads.
//
// One pass over the keys with a running maximum m and sum l per row (logits in
// log2 units, so that one ex2 gives a probability):
//   m' = max(m, max_j x_j),  l' = l 2^(m - m') + sum_j 2^(x_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(x_j - m') v_j,  out = o / l.
//
// A block of 128 threads holds ROWS rows (tokens x query heads of one KV head)
// and walks 64-key tiles; a thread owns 4 rows x 64/TX keys of the logits and
// the same 4 rows x D/TX columns of o, TX = 8 for 64 rows, 32 for 16.  With 64
// rows the work is bound by the FMA pipe: 12 16-byte shared loads feed 128 FMAs
// (as 64 two-wide ones) of the logits, 5 feed 64 of the output at D = 128.  With
// 16 (decode) it is bound by reading the cache.  K of the next tile is on its
// way (cp.async) during the product with V, V of the next during the logits.
// K and V stay in shared memory in their own type; a row is padded by 16 bytes,
// which spreads 8 rows' loads over all banks for every D that is a multiple of 8.
#include <algorithm>
#include <type_traits>

#include "attend.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 64;
constexpr int kSlotRows = 64;
constexpr int kBlocksPerSm = 4;   // at most: the workspace's slots are sized by it

template <typename T>
constexpr int row_bytes(int dim) {
    return dim * (int)sizeof(T) + 16;
}
template <typename T, int ROWS>
size_t smem_bytes(int dim) {
    return (size_t)ROWS * (dim + 4) * 4 + 2 * (size_t)kKeys * row_bytes<T>(dim) +
           (size_t)kKeys * (ROWS + 4) * 4 + (kThreads / 32 + 6) * 8;
}

// Four elements as two pairs.
struct Quad {
    unsigned long long a, b;
};
__device__ __forceinline__ Quad quad(const float *p) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p);
    return {x.x, x.y};
}
__device__ __forceinline__ Quad quad(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return {f2_pack(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)),
            f2_pack(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u))};
}
__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    uint32_t a, b;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(x.w), "f"(x.z));
    *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}

// 16 bytes global -> shared, zeros where !valid (src is then not read).
__device__ __forceinline__ void copy16(void *dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// CT: 16-byte (fp32) column chunks of a thread, CT * TX * 4 >= D.
template <typename T, int ROWS, int CT>
__global__ void __launch_bounds__(kThreads) attend_simt_kernel(const AttendParams p) {
    constexpr int TX = ROWS == 64 ? 8 : 32, KT = kKeys / TX;
    static_assert(TX * (ROWS / 4) == kThreads, "four rows per thread");
    extern __shared__ __align__(16) uint8_t raw[];
    const int D = p.dim, rb = row_bytes<T>(D), vecs = D * (int)sizeof(T) / 16;
    float *sq = reinterpret_cast<float *>(raw);            // [ROWS][D + 4]
    uint8_t *sk = raw + ROWS * (D + 4) * 4;                // [64][rb]
    uint8_t *sv = sk + kKeys * rb;
    float *sp = reinterpret_cast<float *>(sv + kKeys * rb);   // [64 keys][ROWS + 4]
    int64_t *plan = reinterpret_cast<int64_t *>(sp + kKeys * (ROWS + 4));
    uint32_t *s_last = reinterpret_cast<uint32_t *>(plan + kThreads / 32 + 4);
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    const int pr = 1 << p.shift;

    const AttendRun run = attend_plan<kThreads>(p, plan);
    if (run.lo >= run.hi) return;
    int u = run.unit;
    int64_t u_lo = run.unit_lo;
    for (int64_t pos = run.lo; pos < run.hi;) {
        const AttendUnit a = attend_unit(p, u);
        if (a.steps == 0) {
            u = attend_next(p, a, u);
            continue;
        }
        const int64_t end = min(run.hi, u_lo + a.steps);
        const int t0 = (int)(pos - u_lo), t1 = (int)(end - u_lo);
        // eight threads copy a row, 16 rows at a time; pages are looked up
        // ahead of the copies that use them
        int page[4];
        auto look_up = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = t * kKeys + 16 * i + (tid >> 3);
                page[i] = j < a.hi ? attend_page(p, a.list, j >> p.shift) : -1;
            }
        };
        auto fetch = [&](uint8_t *dst, const void *pool, int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * i + (tid >> 3), j = t * kKeys + r;
                const bool valid = page[i] >= 0;
                const T *src = static_cast<const T *>(pool) +
                               (((int64_t)(valid ? page[i] : 0) << p.shift) + (j & (pr - 1))) * D;
                for (int v = tid & 7; v < vecs; v += 8)
                    copy16(dst + r * rb + v * 16, reinterpret_cast<const uint4 *>(src) + v, valid);
            }
            copies_done();
        };
        __syncthreads();   // the unit before is done with shared memory
        look_up(t0);
        fetch(sk, p.k_pool, t0);
        fetch(sv, p.v_pool, t0);
        for (int i = tid; i < ROWS * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            Quad x{0, 0};
            if (r < a.rows) {
                const int token = p.by_group(a.row0 + r), g = a.row0 + r - token * p.group;
                x = quad(static_cast<const T *>(p.q) + (a.q0 + token) * p.q_stride +
                         (int64_t)(a.h * p.group + g) * D + c);
            }
            *reinterpret_cast<ulonglong2 *>(sq + r * (D + 4) + c) = make_ulonglong2(x.a, x.b);
        }
        float m[4], l[4];
        unsigned long long o[4][2 * CT];
        int sees[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            m[i] = -INFINITY;
            l[i] = 0.f;
            sees[i] = r < a.rows ? attend_sees(p, a, r) : 0;
#pragma unroll
            for (int c = 0; c < 2 * CT; ++c) o[i][c] = 0;
        }
        const int sees0 = attend_sees(p, a, 0);
        const bool some = (tid & ~31) / TX * 4 < a.rows;   // the warp has a row
        for (int t = t0; t < t1; ++t) {
            const int j0 = t * kKeys;
            const bool more = t + 1 < t1, edge = j0 + kKeys > sees0;
            copies_wait<1>();
            __syncthreads();   // K and q are here
            if (more) look_up(t + 1);
            if (some) {
                unsigned long long x2[4][KT];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < KT; ++j) x2[i][j] = 0;
                const float *q = sq + ty * 4 * (D + 4);
#pragma unroll 2
                for (int c = 0; c < D; c += 4) {
                    Quad qq[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) qq[i] = quad(q + i * (D + 4) + c);
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        const Quad kk = quad(reinterpret_cast<const T *>(sk + (tx + TX * j) * rb) + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x2[i][j] = f2_fma(qq[i].a, kk.a, x2[i][j]);
                            x2[i][j] = f2_fma(qq[i].b, kk.b, x2[i][j]);
                        }
                    }
                }
                float x[4][KT];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float top = m[i];
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        float lo, hi;
                        f2_unpack(x2[i][j], lo, hi);
                        x[i][j] = (lo + hi) * p.scale_log2;
                        if (edge && j0 + tx + TX * j >= sees[i]) x[i][j] = -INFINITY;
                        top = fmaxf(top, x[i][j]);
                    }
#pragma unroll
                    for (int d = TX / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    // all -inf so far: any finite reference gives 2^-inf = 0
                    const float ref = top == -INFINITY ? 0.f : top;
                    const float down = ex2(m[i] - ref);
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        x[i][j] = ex2(x[i][j] - ref);
                        sum += x[i][j];
                    }
#pragma unroll
                    for (int d = TX / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    l[i] = l[i] * down + sum;
                    m[i] = top;
                    const unsigned long long down2 = f2_pack(down, down);
#pragma unroll
                    for (int c = 0; c < 2 * CT; ++c) o[i][c] = f2_mul(o[i][c], down2);
                }
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    *reinterpret_cast<float4 *>(sp + (tx + TX * j) * (ROWS + 4) + ty * 4) =
                        make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
            }
            __syncthreads();   // K is read, p is here
            if (more)
                fetch(sk, p.k_pool, t + 1);
            else
                copies_done();   // an empty group keeps the count
            copies_wait<1>();
            __syncthreads();   // V is here
            if (some) {
                auto product = [&](auto cut) {
                    const int nk = min(kKeys, a.hi - j0);
#pragma unroll 2
                    for (int j = 0; j < nk; ++j) {
                        const float4 e = *reinterpret_cast<const float4 *>(sp + j * (ROWS + 4) + ty * 4);
                        const unsigned long long e2[4] = {f2_pack(e.x, e.x), f2_pack(e.y, e.y),
                                                          f2_pack(e.z, e.z), f2_pack(e.w, e.w)};
                        const T *v = reinterpret_cast<const T *>(sv + j * rb);
#pragma unroll
                        for (int c = 0; c < CT; ++c) {
                            const int col = (tx + TX * c) * 4;
                            if (CT * TX * 4 == D || col < D) {
                                const Quad vv = quad(v + col);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    // a value that a row does not see may be anything
                                    if (!decltype(cut)::value || j0 + j < sees[i]) {
                                        o[i][2 * c] = f2_fma(e2[i], vv.a, o[i][2 * c]);
                                        o[i][2 * c + 1] = f2_fma(e2[i], vv.b, o[i][2 * c + 1]);
                                    }
                            }
                        }
                    }
                };
                if (edge)
                    product(std::true_type{});
                else
                    product(std::false_type{});
            }
            __syncthreads();   // V and p are read
            if (more)
                fetch(sv, p.v_pool, t + 1);
            else
                copies_done();
        }
        // whole units go straight out, shared ones through the slots
        const bool whole = t0 == 0 && t1 == a.steps;
        const int64_t slot = (int64_t)blockIdx.x * p.slots + (t0 == 0 ? kSlotLast : kSlotFirst);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= a.rows) continue;
            const int64_t row = attend_out_row(p, a, r);
            const float inv = sees[i] > 0 ? 1.f / l[i] : 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int col = (tx + TX * c) * 4;
                if (col >= D) continue;
                float4 y;
                f2_unpack(o[i][2 * c], y.x, y.y);
                f2_unpack(o[i][2 * c + 1], y.z, y.w);
                if (whole) {
                    y = sees[i] > 0 ? make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv)
                                    : make_float4(0, 0, 0, 0);
                    store4(static_cast<T *>(p.out) + row * D + col, y);
                } else {
                    *reinterpret_cast<float4 *>(p.part + (slot * p.slot_rows + r) * D + col) = y;
                }
            }
            if (tx == 0) {
                if (whole)
                    attend_store_lse(p, row, m[i], l[i], sees[i] > 0);
                else
                    p.stat[slot * p.slot_rows + r] = make_float2(m[i], l[i]);
            }
        }
        if (!whole) {
            const int c0 = attend_cta_of(run.total, run.grid, u_lo);
            const int c1 = attend_cta_of(run.total, run.grid, u_lo + a.steps - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool last = atomicAdd(&p.arrived[2 * c0], 1u) == (uint32_t)(c1 - c0);
                if (last) p.arrived[2 * c0] = 0;
                *s_last = last;
            }
            __syncthreads();
            if (*s_last) {
                __threadfence();
                const int chunks = D / 4;
                for (int x = tid; x < a.rows * chunks; x += kThreads) {
                    const int r = x / chunks, col = (x - r * chunks) * 4;
                    auto at = [&](int c) {
                        return ((int64_t)c * p.slots + (c == c0 ? kSlotLast : kSlotFirst)) * p.slot_rows + r;
                    };
                    float top = -INFINITY;
                    for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(&p.stat[at(c)]).x);
                    const float ref = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
                    float4 acc = make_float4(0, 0, 0, 0);
                    for (int c = c0; c <= c1; ++c) {
                        const float2 st = __ldcg(&p.stat[at(c)]);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.part + at(c) * D + col));
                        const float w = ex2(st.x - ref);
                        sum = fmaf(st.y, w, sum);
                        acc.x = fmaf(y.x, w, acc.x);
                        acc.y = fmaf(y.y, w, acc.y);
                        acc.z = fmaf(y.z, w, acc.z);
                        acc.w = fmaf(y.w, w, acc.w);
                    }
                    const bool any = attend_sees(p, a, r) > 0;
                    const int64_t row = attend_out_row(p, a, r);
                    const float inv = 1.f / sum;
                    if (any)
                        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                    else
                        acc = make_float4(0, 0, 0, 0);
                    store4(static_cast<T *>(p.out) + row * D + col, acc);
                    if (col == 0) attend_store_lse(p, row, top, sum, any);
                }
            }
        }
        pos = end;
        u_lo += a.steps;
        u = attend_next(p, a, u);
    }
}

template <typename T, int ROWS, int CT>
int launch(AttendParams &p, int sms, cudaStream_t st) {
    const size_t bytes = smem_bytes<T, ROWS>(p.dim);
    if (bytes > 48 * 1024)
        cudaFuncSetAttribute(attend_simt_kernel<T, ROWS, CT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             232448);
    // as many blocks as an SM holds at once (1 KB of shared memory is each block's own cost)
    static const int by_regs = [] {
        cudaFuncAttributes at{};
        return cudaFuncGetAttributes(&at, attend_simt_kernel<T, ROWS, CT>) == cudaSuccess && at.numRegs > 0
                   ? 65536 / (kThreads * ((at.numRegs + 7) / 8 * 8)) : 1;
    }();
    const int per_sm = std::max(1, std::min({kBlocksPerSm, by_regs, (int)(233472 / (bytes + 1024))}));
    attend_simt_kernel<T, ROWS, CT><<<per_sm * sms, kThreads, bytes, st>>>(p);
    return cache_launched("kvc_attend");
}

template <typename T>
int launch_type(AttendParams &p, int rows, int sms, cudaStream_t st) {
    const int d = p.dim;
    if (rows == 16) return d <= 128 ? launch<T, 16, 1>(p, sms, st) : launch<T, 16, 2>(p, sms, st);
    return d <= 64    ? launch<T, 64, 2>(p, sms, st)
           : d <= 96  ? launch<T, 64, 3>(p, sms, st)
           : d <= 128 ? launch<T, 64, 4>(p, sms, st)
                      : launch<T, 64, 8>(p, sms, st);
}

}  // namespace

AttendNeeds attend_simt_needs(int sms) { return {kBlocksPerSm * sms, 2, kSlotRows}; }

int launch_attend_simt(AttendParams &p, bool f32, int grid, cudaStream_t st) {
    // 16 rows per block where a list's tokens fill no more
    const int rows = p.max_new * p.group <= 16 ? 16 : 64;
    if (!attend_units(p, rows)) {
        set_error("kvc_attend: n_seqs * n_kv_heads * max_new is too large");
        return KVC_ERR_UNSUPPORTED;
    }
    p.step_keys = kKeys;
    p.split_rows = 0;
    const int sms = grid / kBlocksPerSm;
    return f32 ? launch_type<float>(p, rows, sms, st) : launch_type<__nv_bfloat16>(p, rows, sms, st);
}

}  // namespace kvc
