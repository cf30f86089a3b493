// attend_pieces.cuh -- attention of many rows over a cache held in 4 or 8 bits where
// tcgen05's kernel does not reach: fp32, other head sizes than 64 and 128, and groups
// of more than 128 query heads.  (Lists of up to 16 rows are attend_simt.cuh's.)
//
// The formulas are attend_simt.cuh's, to fp32's accuracy, on the tensor instruction of
// a warp (mma.m16n8k16).  What a code of a row of K or V stands for is exact in bf16;
// an fp32 number of Q or P is the sum of three bf16 numbers, exactly:
//   x1 = x cut off after 8 significant bits,  x2 = x - x1 cut off so,  x3 = x - x1 - x2,
// so a product is three, each of whose terms fits fp32; they are summed there.  Rows of
// bf16 are one piece of Q, but three of P.  The tensor instruction drops bits of its sums
// toward zero, so chains of it are kept short: the first pieces' sums go apart from the
// others', whose lost bits are then 2^-8 as large, and every tile's start anew and are
// added to the tiles' before in fp32.  The outputs' error against 64 bits is then 1.9e-7
// of their norm (in one chain each 1.2e-6 to 3.4e-6, more the longer the lists; elementary
// fp32 operations 6e-7 to 1e-6), for 4% of the time.
//
// 64 rows to a block, 16 to a warp; a tile of 64 keys comes to shared memory as it is
// held and is written out from there as bf16; P never leaves the registers.  A value of
// V that stands for NaN is written as zero, for the sake of the rows that do not see
// it, and those that do become NaN by themselves.
//
// The products are three times the algorithmic ones and run at a fifth of the tensor
// pipe's time; what bounds it is the chain of a tile (writing it out, product, softmax,
// product) with twelve warps on an SM to hide it: issue slots are a third used.  Five
// chunks of up to 301 tokens x 8 heads of 80 in fp32 over up to 2,700 rows in 4 bits: 69
// us, 41 TFLOP/s of algorithmic work; the CUDA cores took 139, and they take 121 over
// rows in fp32.
#pragma once

#include "attend_simt.cuh"

namespace kvc {

namespace {

constexpr int kPieceRows = 64, kPieceKeys = 64, kPieceThreads = 128;

// Columns in shared memory, of whole tensor instructions; their bytes, padded so that
// ldmatrix meets all banks.
__host__ __device__ constexpr int piece_cols(int dim) { return (dim + 15) / 16 * 16; }
__host__ __device__ constexpr int piece_row(int dim) { return piece_cols(dim) * 2 + 16; }
template <typename T>
constexpr int pieces_of() {
    return sizeof(T) == 4 ? 3 : 1;
}
template <typename T, int BITS>
size_t piece_smem(int dim) {
    const size_t held = (size_t)kPieceKeys / kQuantRows * quant_block(BITS, quant_groups(dim));
    return (size_t)(pieces_of<T>() * kPieceRows + 2 * kPieceKeys) * piece_row(dim) + 2 * held + (kPieceThreads / 32 + 6) * 8;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_turned(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The upper halves of two words: two numbers cut off after 8 significant bits.
__device__ __forceinline__ uint32_t upper(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float rest(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// The pieces of two numbers.
__device__ __forceinline__ void cut(float x, float y, uint32_t (&piece)[3]) {
    const float x2 = rest(x), y2 = rest(y);
    piece[0] = upper(x, y);
    piece[1] = upper(x2, y2);
    piece[2] = upper(rest(x2), rest(y2));
}

// KS steps of 16 columns hold a row.  Blocks per SM: 168 registers a thread do not hold
// the sums of 128 columns (8 heads of 128: 104 us with three blocks, 92 with two).
constexpr int piece_blocks(int ks) { return ks <= 6 ? 3 : 2; }
template <typename T, int KS, int BITS>
__global__ void __launch_bounds__(kPieceThreads, piece_blocks(KS)) attend_pieces_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kThreads = kPieceThreads, kPieces = pieces_of<T>(), kBlocks = kPieceKeys / kQuantRows;
    extern __shared__ __align__(16) uint8_t raw[];
    const int D = p.dim, rb = piece_row(D), steps = piece_cols(D) / 16, groups = quant_groups(D), block = quant_block(BITS, groups);
    uint8_t *sq = raw;                                     // [piece][64][rb]
    uint8_t *sk = sq + kPieces * kPieceRows * rb;          // [64][rb]
    uint8_t *sv = sk + kPieceKeys * rb;
    uint8_t *hk = sv + kPieceKeys * rb;                    // rows as they are held
    uint8_t *hv = hk + kBlocks * block;
    int64_t *plan = reinterpret_cast<int64_t *>(hv + kBlocks * block);
    uint32_t *s_last = reinterpret_cast<uint32_t *>(plan + kThreads / 32 + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c = lane & 3;
    const int pr = 1 << p.shift;
    // what the lane addresses for ldmatrix: 16 rows of Q (K's first columns, then the
    // next), 16 keys of K (8 by 16 columns), 16 keys of V
    const uint32_t q_at = smem_u32(sq) + (16 * warp + (lane & 15)) * rb + 16 * (lane >> 4);
    const uint32_t k_at = smem_u32(sk) + ((lane & 7) + (lane >> 4 << 3)) * rb + 16 * (lane >> 3 & 1);
    const uint32_t v_at = smem_u32(sv) + (lane & 15) * rb + 16 * (lane >> 4);

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
        const int64_t end = min(run.hi, u_lo + a.cost);
        const int t0 = max(0, (int)(pos - u_lo) - p.extra), t1 = max(0, (int)(end - u_lo) - p.extra);
        if (t1 <= t0) {   // nothing but what the unit costs beside its steps
            pos = end;
            if (end == u_lo + a.cost) {
                u_lo += a.cost;
                u = attend_next(p, a, u);
            }
            continue;
        }
        int page[kBlocks];   // of the tile's blocks, looked up ahead of the copies that use them
        auto look_up = [&](int t) {
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const int j = t * kPieceKeys + kQuantRows * i;
                page[i] = j < a.hi ? attend_page(p, a.list, j >> p.shift) : -1;
            }
        };
        auto fetch = [&](uint8_t *dst, const void *pool, int t) {
            const int per = block / 16;
            for (int v = tid; v < kBlocks * per; v += kThreads) {
                const int i = (v >= per) + (v >= 2 * per) + (v >= 3 * per), j = t * kPieceKeys + kQuantRows * i;
                const int pg = i < 2 ? (i == 0 ? page[0] : page[1]) : (i == 2 ? page[2] : page[3]);
                const bool valid = pg >= 0;
                const uint8_t *src =
                    static_cast<const uint8_t *>(pool) + ((((int64_t)(valid ? pg : 0) << p.shift) + (j & (pr - 1))) >> 4) * block;
                copy16(dst + v * 16, src + (v - i * per) * 16, valid);
            }
            copies_done();
        };
        // held rows to a tile, eight threads a row; rows past the last key and groups of
        // V that stand for NaN as zeros.  Whether there are such.
        auto write_out = [&](uint8_t *dst, const uint8_t *held, int nk, bool of_v) {
            bool odd = false;
#pragma unroll 2
            for (int r = tid >> 3; r < kPieceKeys; r += kThreads / 8) {
                const QuantRow at = quant_row(BITS, groups, r);
                for (int e = tid & 7; e < 2 * steps; e += 8) {
                    const uint32_t word = reinterpret_cast<const uint16_t *>(held + at.words)[e >> 2];
                    uint32_t y[4];
                    quant_bf16<BITS>(quant_load<BITS>(held + at.codes, groups, e >> 2, e & 3, of_v), word * 0x10001u, y);
                    const bool none = quant_is_nan<BITS>(word);
                    odd |= of_v && none && r < nk;
                    const uint32_t is = r < nk && !(of_v && none) ? 0xffffffffu : 0;
                    *reinterpret_cast<uint4 *>(dst + r * rb + 16 * e) = make_uint4(y[0] & is, y[1] & is, y[2] & is, y[3] & is);
                }
            }
            return odd;
        };
        __syncthreads();   // the unit before is done with shared memory
        look_up(t0);
        fetch(hk, p.k_pool, t0);
        fetch(hv, p.v_pool, t0);
        for (int i = tid; i < kPieceRows * 4 * steps; i += kThreads) {   // four columns each
            const int r = i / (4 * steps), col = (i - r * (4 * steps)) * 4;
            const int token = p.by_group(a.row0 + r), g = a.row0 + r - token * p.group;
            const bool there = r < a.rows && col < D;
            const T *src = static_cast<const T *>(p.q) + (a.q0 + token) * p.q_stride + (int64_t)(a.h * p.group + g) * D + col;
            uint8_t *dst = sq + r * rb + col * 2;
            if constexpr (kPieces == 1) {
                *reinterpret_cast<uint2 *>(dst) = there ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0, 0);
            } else {
                const float4 x = there ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                uint32_t lo[3], hi[3];
                cut(x.x, x.y, lo);
                cut(x.z, x.w, hi);
                // an infinity is its first piece alone
                const bool fx = isinf(x.x), fy = isinf(x.y), fz = isinf(x.z), fw = isinf(x.w);
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    if (e > 0) {
                        lo[e] &= (fx ? 0xffff0000u : 0xffffffffu) & (fy ? 0xffffu : 0xffffffffu);
                        hi[e] &= (fz ? 0xffff0000u : 0xffffffffu) & (fw ? 0xffffu : 0xffffffffu);
                    }
                    *reinterpret_cast<uint2 *>(dst + e * kPieceRows * rb) = make_uint2(lo[e], hi[e]);
                }
            }
        }
        // of rows 16 warp + r8 and + 8 more
        float m[2], l[2], o[2 * KS][4];
        int sees[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * warp + r8 + 8 * i;
            m[i] = -INFINITY;
            l[i] = 0.f;
            sees[i] = r < a.rows ? attend_sees(p, a, r) : 0;
        }
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        const int sees0 = attend_sees(p, a, 0);   // the fewest
        const bool some = 16 * warp < a.rows;     // the warp has a row
        for (int t = t0; t < t1; ++t) {
            const int j0 = t * kPieceKeys, nk = min(kPieceKeys, a.hi - j0);
            const bool more = t + 1 < t1;
            if (more) look_up(t + 1);
            copies_wait<0>();
            __syncthreads();   // the rows are here, the tiles before are read
            write_out(sk, hk, nk, false);
            const bool odd = __syncthreads_or(write_out(sv, hv, nk, true));
            if (more) {
                fetch(hk, p.k_pool, t + 1);
                if (!odd) fetch(hv, p.v_pool, t + 1);
            }
            if (some) {
                float x[kPieceKeys / 8][4];
#pragma unroll
                for (int half = 0; half < 2; ++half) {   // 32 keys at a time
                    float small[4][4];   // sums of the later pieces; x: of the first
#pragma unroll
                    for (int n = 0; n < 16; ++n) x[4 * half + (n >> 2)][n & 3] = small[n >> 2][n & 3] = 0.f;
#pragma unroll 1
                    for (int s = 0; s < steps; ++s) {
                        uint32_t q[kPieces][4], k[2][4];
#pragma unroll
                        for (int e = 0; e < kPieces; ++e) ldmatrix4(q[e], q_at + e * kPieceRows * rb + 32 * s);
#pragma unroll
                        for (int n = 0; n < 2; ++n) ldmatrix4(k[n], k_at + (32 * half + 16 * n) * rb + 32 * s);
#pragma unroll
                        for (int e = kPieces - 1; e >= 0; --e)
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                mma_bf16(e == 0 ? x[4 * half + n] : small[n], q[e], k[n >> 1][2 * (n & 1)], k[n >> 1][2 * (n & 1) + 1]);
                    }
#pragma unroll
                    for (int n = 0; n < 16; ++n) x[4 * half + (n >> 2)][n & 3] += small[n >> 2][n & 3];
                }
                const bool edge = j0 + kPieceKeys > sees0;
                float downs[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = m[i];
#pragma unroll
                    for (int n = 0; n < kPieceKeys / 8; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &y = x[n][2 * i + h];
                            y *= p.scale_log2;
                            if (edge && j0 + 8 * n + 2 * c + h >= sees[i]) y = -INFINITY;
                            top = fmaxf(top, y);
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // all -inf so far: any finite reference gives 2^-inf = 0
                    const float ref = top == -INFINITY ? 0.f : top;
                    const float down = ex2(m[i] - ref);
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < kPieceKeys / 8; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &y = x[n][2 * i + h];
                            y = ex2(y - ref);
                            sum += y;
                        }
                    l[i] = l[i] * down + sum;   // (the lane's share)
                    m[i] = top;
                    downs[i] = down;
                }
                uint32_t e[kPieceKeys / 16][3][4];
#pragma unroll
                for (int s = 0; s < kPieceKeys / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t y[3];
                        cut(x[2 * s + (i >> 1)][2 * (i & 1)], x[2 * s + (i >> 1)][2 * (i & 1) + 1], y);
                        e[s][0][i] = y[0];
                        e[s][1][i] = y[1];
                        e[s][2][i] = y[2];
                    }
#pragma unroll
                for (int n = 0; n < KS; ++n) {
                    if (n >= steps) continue;
                    float sum[2][4], small[2][4];
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i >> 2][i & 3] = small[i >> 2][i & 3] = 0.f;
#pragma unroll
                    for (int s = 0; s < kPieceKeys / 16; ++s) {
                        uint32_t v[4];
                        ldmatrix4_turned(v, v_at + 16 * s * rb + 32 * n);
#pragma unroll
                        for (int i = 2; i >= 0; --i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) mma_bf16(i == 0 ? sum[h] : small[h], e[s][i], v[2 * h], v[2 * h + 1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[2 * n + h][i] = fmaf(o[2 * n + h][i], downs[i >> 1], sum[h][i] + small[h][i]);
                }
            }
            if (odd) {
                if (some)
                    for (int j = 0; j < nk; ++j) {
                        const uint16_t *words = reinterpret_cast<const uint16_t *>(hv + quant_row(BITS, groups, j).words);
#pragma unroll
                        for (int g = 0; g < (KS + 1) / 2; ++g)
                            if (g < groups && quant_is_nan<BITS>(words[g]))
#pragma unroll
                                for (int n = 4 * g; n < min(4 * g + 4, 2 * KS); ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        if (j0 + j < sees[i >> 1]) o[n][i] = __int_as_float(0x7fffffff);
                    }
                __syncthreads();   // V's words are read
                if (more) fetch(hv, p.v_pool, t + 1);
            }
        }
        // whole units go straight out, shared ones through the slots
        const bool whole = t0 == 0 && t1 == a.steps;
        const int64_t slot = (int64_t)blockIdx.x * p.slots + (t0 == 0 ? kSlotLast : kSlotFirst);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            const int r = 16 * warp + r8 + 8 * i;
            if (r >= a.rows) continue;
            const int64_t row = attend_out_row(p, a, r);
            const float inv = sees[i] > 0 ? 1.f / l[i] : 0.f;
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
                const int col = 8 * n + 2 * c;
                if (8 * n >= D) continue;
                const float y0 = o[n][2 * i], y1 = o[n][2 * i + 1];
                if (whole)
                    store2(static_cast<T *>(p.out) + row * D + col, sees[i] > 0 ? y0 * inv : 0.f, sees[i] > 0 ? y1 * inv : 0.f);
                else
                    store2(p.part + (slot * p.slot_rows + r) * D + col, y0, y1);
            }
            if (c == 0) {
                if (whole)
                    attend_store_lse(p, row, m[i], l[i], sees[i] > 0);
                else
                    p.stat[slot * p.slot_rows + r] = make_float2(m[i], l[i]);
            }
        }
        if (!whole) attend_meet<T, kThreads>(p, run, a, u_lo, s_last);
        pos = end;
        u_lo += a.cost;
        u = attend_next(p, a, u);
    }
}

template <typename T, int KS, int BITS>
int launch_pieces_of(AttendParams &p, int sms, cudaStream_t st) {
    constexpr auto kernel = attend_pieces_kernel<T, KS, BITS>;
    const size_t bytes = piece_smem<T, BITS>(p.dim);
    if (bytes > 48 * 1024) allow_shared<kernel>(232448);
    // as many blocks as an SM holds at once (1 KB of shared memory is each block's own cost)
    const int per_sm = std::max(1, std::min(piece_blocks(KS), (int)(233472 / (bytes + 1024))));
    launch_early(kernel, per_sm * sms, kPieceThreads, bytes, st, p);
    return cache_launched(attend_name(p));
}

template <typename T, int BITS>
int launch_pieces(AttendParams &p, int sms, cudaStream_t st) {
    const int d = p.dim;
    return d <= 64    ? launch_pieces_of<T, 4, BITS>(p, sms, st)
           : d <= 96  ? launch_pieces_of<T, 6, BITS>(p, sms, st)
           : d <= 128 ? launch_pieces_of<T, 8, BITS>(p, sms, st)
                      : launch_pieces_of<T, 16, BITS>(p, sms, st);
}

}  // namespace

}  // namespace kvc
