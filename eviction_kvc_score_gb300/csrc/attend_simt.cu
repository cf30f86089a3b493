// attend_simt.cu -- attention of new tokens over the paged cache on the CUDA
// cores, fp32 throughout: fp32 caches, head sizes the tensor cores' kernel does
// not take, and groups of more than 128 query heads.
//
// One pass over the keys with a running maximum m and sum l per row (logits in
// log2 units, so that one ex2 gives a probability):
//   m' = max(m, max_j x_j),  l' = l 2^(m - m') + sum_j 2^(x_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(x_j - m') v_j,  out = o / l.
//
// A block holds ROWS rows (tokens x query heads of one KV head) and walks 64-key
// tiles; a thread owns 4 rows x 64/TX keys of the logits and the same 4 rows x
// D/TX columns of o: 256 threads, TX = 16 for 64 rows; 128 threads, TX = 32 for
// 16 rows.  With 64 rows the work is bound by the FMA pipe, with 16 (decode) by
// reading the cache.  (Tiles of 4 x 8 keys by 128 threads need fewer shared
// loads but 250 registers: eight warps per SM left the FMA pipe at a third, 179 us
// for five chunks of up to 293 tokens x 8 heads of 80 over up to 2,757 rows; now 120
// us, 24 TFLOP/s, FMA pipe and shared loads each half busy.  Decode of 2 x 4 lists
// of 60,000 rows: 120 us, 4.1 TB/s.)  K of the next tile is on its
// way (cp.async) during the product with V, V of the next during the logits.
// K and V stay in shared memory in their own type; a row is padded by 16 bytes,
// which spreads 8 rows' loads over all banks for every D that is a multiple of 8.
#include <algorithm>
#include <type_traits>

#include "attend.cuh"

namespace kvc {

namespace {

constexpr int kKeys = 64;
constexpr int kSlotRows = 64;
constexpr int kBlocksPerSm = 4;   // at most: the workspace's slots are sized by it

template <typename T>
constexpr int row_bytes(int dim) {
    return dim * (int)sizeof(T) + 16;
}
constexpr int threads_of(int rows) { return rows == 64 ? 256 : 128; }
template <typename T, int ROWS>
size_t smem_bytes(int dim) {
    return (size_t)ROWS * (dim + 4) * 4 + 2 * (size_t)kKeys * row_bytes<T>(dim) +
           (size_t)kKeys * (ROWS + 4) * 4 + (threads_of(ROWS) / 32 + 6) * 8;
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
template <int N>
struct Pairs {
    unsigned long long v[N];
};
// 2 N elements as N pairs, N = 1 or 2.
template <int N, typename T>
__device__ __forceinline__ Pairs<N> pairs_at(const T *p) {
    Pairs<N> r;
    if constexpr (N == 2) {
        const Quad q = quad(p);
        r.v[0] = q.a;
        r.v[1] = q.b;
    } else if constexpr (sizeof(T) == 4) {
        r.v[0] = *reinterpret_cast<const unsigned long long *>(p);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        r.v[0] = f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    return r;
}
__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) {
    uint32_t a;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(y), "f"(x));
    *reinterpret_cast<uint32_t *>(p) = a;
}
// Whether the 16 bytes at p hold numbers only.
__device__ __forceinline__ bool all_finite(const float *p) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    return isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w);
}
__device__ __forceinline__ bool all_finite(const __nv_bfloat16 *p) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    const uint32_t low = __vminu2(__vminu2(~x.x & 0x7f807f80u, ~x.y & 0x7f807f80u),
                                  __vminu2(~x.z & 0x7f807f80u, ~x.w & 0x7f807f80u));
    return (low & 0xffffu) != 0 && (low >> 16) != 0;
}

// 16 bytes global -> shared, zeros where !valid (src is then not read).
__device__ __forceinline__ void copy16(void *dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The block's rows of a slot are written: count it; true in the whole block if it
// is the last of `all` (one alone is not counted, as in attend_last).
__device__ __forceinline__ bool block_last(uint32_t *count, uint32_t all, uint32_t *s_last) {
    __threadfence();
    __syncthreads();
    if (all == 1) return true;
    if (threadIdx.x == 0) {
        const bool last = atomicAdd(count, 1u) == all - 1;
        if (last) *count = 0;
        *s_last = last;
    }
    __syncthreads();
    const bool last = *s_last;
    __threadfence();
    return last;
}

// A thread's columns: CT chunks of 2 N, CT * TX * 2 N >= D.
template <typename T, int ROWS, int N, int CT>
__global__ void __launch_bounds__(threads_of(ROWS), ROWS == 64 ? 2 : 4) attend_simt_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kThreads = threads_of(ROWS), W = 2 * N;
    constexpr int TX = ROWS == 64 ? 16 : 32, KT = kKeys / TX;
    constexpr int kPass = kThreads / 8, kPasses = kKeys / kPass;   // rows copied at a time
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

    let_next_start();
    wait_for_inputs();
    const AttendRun run = attend_plan<kThreads, true>(p, plan);
    if (run.lo >= run.hi) return;
    int u = run.unit;
    int64_t u_lo = run.unit_lo;
    for (int64_t pos = run.lo; pos < run.hi;) {
        const AttendUnit a = attend_unit<true>(p, u);
        if (a.steps == 0) {
            u = attend_next_seq<true>(p, a.b);
            continue;
        }
        const int64_t end = min(run.hi, u_lo + a.steps);
        const int t0 = (int)(pos - u_lo), t1 = (int)(end - u_lo);
        // eight threads copy a row; pages are looked up ahead of the copies
        // that use them
        int page[kPasses];
        auto look_up = [&](int t) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int j = t * kKeys + kPass * i + (tid >> 3);
                page[i] = j < a.hi ? attend_page(p, a.list, j >> p.shift) : -1;
            }
        };
        auto fetch = [&](uint8_t *dst, const void *pool, int t) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = kPass * i + (tid >> 3), j = t * kKeys + r;
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
        unsigned long long o[4][N * CT];
        int sees[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            m[i] = -INFINITY;
            l[i] = 0.f;
            sees[i] = r < a.rows ? attend_sees(p, a, r) : 0;
#pragma unroll
            for (int c = 0; c < N * CT; ++c) o[i][c] = 0;
        }
        const int sees0 = attend_sees(p, a, 0);
        copies_wait<1>();
        __syncthreads();   // the first K and q are here
        const bool some = (tid & ~31) / TX * 4 < a.rows;   // the warp has a row
        for (int t = t0; t < t1; ++t) {
            const int j0 = t * kKeys;
            const bool more = t + 1 < t1, edge = j0 + kKeys > sees0;
            if (more) look_up(t + 1);
            if (some) {
                unsigned long long x2[4][KT];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < KT; ++j) x2[i][j] = 0;
                const float *q = sq + ty * 4 * (D + 4);
#pragma unroll 4
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
                    for (int c = 0; c < N * CT; ++c) o[i][c] = f2_mul(o[i][c], down2);
                }
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    *reinterpret_cast<float4 *>(sp + (tx + TX * j) * (ROWS + 4) + ty * 4) =
                        make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
            }
            copies_wait<0>();
            __syncthreads();   // K is read, p and V are here
            if (more) fetch(sk, p.k_pool, t + 1);
            const int nk = min(kKeys, a.hi - j0);
            // where some row sees only part of the tile, p is 0 for the rest,
            // but 0 times an infinite or NaN value is not
            bool strict = false;
            if (edge) {
                bool odd = false;
                for (int r = max(0, sees0 - j0) + (tid >> 3); r < nk; r += kPass)
                    for (int v = tid & 7; v < vecs; v += 8)
                        odd |= !all_finite(reinterpret_cast<const T *>(sv + r * rb + v * 16));
                strict = __syncthreads_or(odd);
            }
            if (some) {
                auto product = [&](auto cut) {
#pragma unroll 4
                    for (int j = 0; j < nk; ++j) {
                        const float4 e = *reinterpret_cast<const float4 *>(sp + j * (ROWS + 4) + ty * 4);
                        const unsigned long long e2[4] = {f2_pack(e.x, e.x), f2_pack(e.y, e.y),
                                                          f2_pack(e.z, e.z), f2_pack(e.w, e.w)};
                        const T *v = reinterpret_cast<const T *>(sv + j * rb);
#pragma unroll
                        for (int c = 0; c < CT; ++c) {
                            // columns past D are read from the row's end on (still
                            // shared memory) and never stored
                            const Pairs<N> vv = pairs_at<N>(v + (tx + TX * c) * W);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                // a value that a row does not see may be anything
                                if (!decltype(cut)::value || j0 + j < sees[i])
#pragma unroll
                                    for (int h = 0; h < N; ++h)
                                        o[i][N * c + h] = f2_fma(e2[i], vv.v[h], o[i][N * c + h]);
                        }
                    }
                };
                if (strict)
                    product(std::true_type{});
                else
                    product(std::false_type{});
            }
            if (more) {
                copies_wait<0>();
                __syncthreads();   // V and p are read, the next K is here
                fetch(sv, p.v_pool, t + 1);
            }
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
            for (int c = 0; c < N * CT; ++c) {
                const int col = (tx + TX * (c / N)) * W + 2 * (c % N);
                if (col >= D) continue;
                float y0, y1;
                f2_unpack(o[i][c], y0, y1);
                if (whole)
                    store2(static_cast<T *>(p.out) + row * D + col, sees[i] > 0 ? y0 * inv : 0.f,
                           sees[i] > 0 ? y1 * inv : 0.f);
                else
                    store2(p.part + (slot * p.slot_rows + r) * D + col, y0, y1);
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
            const int me = blockIdx.x, n = c1 - c0 + 1, groups = attend_groups(n);
            bool last = true;
            if (groups > 1) {
                const int g0 = c0 + (me - c0) / kJoinGroup * kJoinGroup, gn = min(kJoinGroup, c1 - g0 + 1);
                last = block_last(&p.arrived[16 * g0 + 8], gn, s_last);
                if (last) attend_join<T, 2, 4>(p, a, AttendSpan{c0, g0, 1, gn, false, false}, 0, a.rows, 0, tid, kThreads);
            }
            if (last && block_last(&p.arrived[16 * c0], groups > 1 ? groups : n, s_last))
                attend_join<T, 2, 4>(p, a, AttendSpan{c0, c0, groups > 1 ? kJoinGroup : 1, groups > 1 ? groups : n, groups > 1, true},
                                     0, a.rows, 0, tid, kThreads);
        }
        pos = end;
        u_lo += a.steps;
        u = attend_next(p, a, u);
    }
}

template <typename T, int ROWS, int N, int CT>
int launch(AttendParams &p, int sms, cudaStream_t st) {
    constexpr auto kernel = attend_simt_kernel<T, ROWS, N, CT>;
    const size_t bytes = smem_bytes<T, ROWS>(p.dim);
    if (bytes > 48 * 1024) allow_shared<kernel>(232448);
    // as many blocks as an SM holds at once (1 KB of shared memory is each block's own cost)
    const int per_sm = std::max(1, std::min(ROWS == 64 ? 2 : 4, (int)(233472 / (bytes + 1024))));
    launch_early(kernel, per_sm * sms, threads_of(ROWS), bytes, st, p);
    return cache_launched("kvc_attend");
}

template <typename T>
int launch_type(AttendParams &p, int rows, int sms, cudaStream_t st) {
    const int d = p.dim;
    if (rows == 16)
        return d <= 64    ? launch<T, 16, 1, 1>(p, sms, st)
               : d <= 128 ? launch<T, 16, 2, 1>(p, sms, st)
                          : launch<T, 16, 2, 2>(p, sms, st);
    return d <= 64    ? launch<T, 64, 2, 1>(p, sms, st)
           : d <= 96  ? launch<T, 64, 1, 3>(p, sms, st)
           : d <= 128 ? launch<T, 64, 2, 2>(p, sms, st)
           : d <= 192 ? launch<T, 64, 2, 3>(p, sms, st)
                      : launch<T, 64, 2, 4>(p, sms, st);
}

}  // namespace

AttendNeeds attend_simt_needs(int sms) { return {kBlocksPerSm * sms, 2, kSlotRows}; }

int launch_attend_simt(AttendParams &p, bool f32, int grid, cudaStream_t st) {
    p.step_keys = kKeys;
    p.split_rows = 0;
    p.extra = 0;
    const int sms = grid / kBlocksPerSm;
    // Blocks of 64 rows, of 16 where no list has more.  Lists of both kinds take a
    // launch each: in a block of 64 rows one warp of eight would work on a token's
    // (a chunk of 256 tokens and 255 decoding sequences of 1,000 rows, fp32, 8 KV
    // heads of 128: 2,512 us in one launch, 1,035 in two).  A launch that finds no
    // list costs 6 us, so one does where the lists have more than 128 rows on
    // average: the short ones are then at most a third of the blocks.
    const int64_t most = (int64_t)p.max_new * p.group;
    const bool both = most > 16 && p.group <= 16 && p.n_tokens * p.group <= 128 * (int64_t)p.n_seqs;
    for (int rows = most > 16 ? 64 : 16; rows >= 16; rows -= both ? 48 : rows) {
        const bool large = rows == 64;
        if (!attend_units(p, rows, large && both ? 16 : 0, large ? INT_MAX : 16)) {
            set_error("kvc_attend: n_seqs * n_kv_heads * max_new is too large");
            return KVC_ERR_UNSUPPORTED;
        }
        const int rc = f32 ? launch_type<float>(p, rows, sms, st) : launch_type<__nv_bfloat16>(p, rows, sms, st);
        if (rc) return rc;
    }
    return KVC_OK;
}

}  // namespace kvc
