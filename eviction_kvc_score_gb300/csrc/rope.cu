// rope.cu -- rotary positions of new tokens' queries and keys, and of kept
// keys that move to other positions.
//
// A pair (a, b) of a head at position p turns by the angle 2 pi p u, u turns
// per position.  u is held as a 64-bit fraction, and the product with the
// integer p modulo 2^64 IS the angle modulo a full turn, exactly: no position
// is too far and the reduction is one integer multiply.  What is left is a
// quarter turn and one sincospi of at most an eighth of a turn either way, whose
// rounding to fp32 moves the angle by pi 2^-27 at most.
//
// Each block takes a few tokens, computes every (token, pair) angle once into
// shared memory and turns all their heads with 16-byte loads and stores.  Bound
// by HBM: 32,768 tokens of 32 + 8 heads of 128 (bf16, out of place, 671 MB) take
// 106-107 us, 6.3 TB/s or 93% of the measured copy rate; 64 tokens 2.7 us, mostly
// launch.
#include <algorithm>

#include "cache.cuh"

namespace kvc {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kTableThreads = 32;  // a warp per SM: fp64 instructions are issued rarely
constexpr int kRopePairs = 512;   // (token, pair) angles of a block

// A number as the unevaluated sum h + l, |l| <= ulp(h) / 2: about 106 bits
// (Dekker, "A floating-point technique for extending the available precision",
// 1971).  A double's 53 bits would leave the last 11 of the table's 64 empty,
// 2.6e-7 rad at position 2^31.
struct Twice {
    double h, l;
};
__device__ Twice exact_sum(double a, double b) {
    const double s = __dadd_rn(a, b), t = __dsub_rn(s, a);
    return {s, __dadd_rn(__dsub_rn(a, __dsub_rn(s, t)), __dsub_rn(b, t))};
}
__device__ Twice exact_product(double a, double b) {
    const double p = __dmul_rn(a, b);
    return {p, __fma_rn(a, b, -p)};
}
__device__ Twice operator+(Twice a, Twice b) {
    const Twice s = exact_sum(a.h, b.h);
    return exact_sum(s.h, __dadd_rn(s.l, __dadd_rn(a.l, b.l)));
}
__device__ Twice operator*(Twice a, Twice b) {
    const Twice p = exact_product(a.h, b.h);
    return exact_sum(p.h, __dadd_rn(p.l, __fma_rn(a.h, b.l, __dmul_rn(a.l, b.h))));
}
__device__ Twice operator-(Twice a) { return {-a.h, -a.l}; }
__device__ Twice operator/(Twice a, Twice b) {   // long division, a quotient's double at a time
    const double q0 = a.h / b.h;
    const Twice r = a + -(Twice{q0, 0} * b);
    const double q1 = r.h / b.h;
    const Twice left = r + -(Twice{q1, 0} * b);
    return exact_sum(q0, q1) + Twice{left.h / b.h, 0};
}
__device__ Twice scaled(Twice a, int by) { return {ldexp(a.h, by), ldexp(a.l, by)}; }

__device__ Twice ln2() { return {0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56}; }
__device__ Twice half_over_pi() { return {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57}; }
// 1 / n, for the compiler to work out.
__device__ __forceinline__ Twice inverse(int n) {
    const double h = 1.0 / n;
    return {h, fma(-(double)n, h, 1.0) / n};
}

// e^x, |x| < 710: x = k ln 2 + 256 t, |t| < 0.0014, the series of e^t - 1 up to
// t^7 (t^8 / 8! is 2^-91) and 2^k (1 + it)^256 by doubling, (1 + y)^2 = 1 + (2 y + y^2).
__device__ Twice exponential(Twice x) {
    const double k = rint(x.h / ln2().h);
    const Twice t = scaled(x + -(Twice{k, 0} * ln2()), -8);
    Twice y = t * inverse(7);
#pragma unroll
    for (int n = 6; n >= 1; --n) y = t * (Twice{1, 0} + y) * inverse(n);
#pragma unroll
    for (int n = 0; n < 8; ++n) y = scaled(y, 1) + y * y;
    return scaled(Twice{1, 0} + y, (int)k);
}
// The root of e^y = m near log(m): y + (m e^-y - 1).
__device__ Twice logarithm(double x) {
    int e;
    const double m = frexp(x, &e);
    const Twice y{log(m), 0};
    return Twice{(double)e, 0} * ln2() + y + (Twice{m, 0} * exponential(-y) + Twice{-1, 0});
}

__global__ void rope_table_kernel(int rot, double theta, double factor, double alpha, double beta,
                                  double context, uint64_t *table) {
    const int i = blockIdx.x * kTableThreads + threadIdx.x;
    if (i >= rot / 2) return;
    const Twice power = Twice{-2.0 * i, 0} / Twice{(double)rot, 0};
    Twice f = exponential(power * logarithm(theta)) * half_over_pi();   // turns per position
    if (factor > 1.0) {
        const Twice turns = f * Twice{context, 0};
        Twice g;
        if (turns.h > beta || (turns.h == beta && turns.l >= 0.0))
            g = {1, 0};
        else if (turns.h < alpha || (turns.h == alpha && turns.l <= 0.0) || isinf(beta))
            g = {0, 0};
        else
            g = (turns + Twice{-alpha, 0}) / exact_sum(beta, -alpha);
        f = f * (g + (Twice{1, 0} + -g) / Twice{factor, 0});
    }
    // to the nearest 2^-64: what h has of whole units, then the rest
    const double units = f.h * 0x1p64, whole = floor(units);
    table[i] = (uint64_t)whole + (uint64_t)(int64_t)rint((units - whole) + f.l * 0x1p64);
}

struct RopeSide {
    const void *x;
    void *y;
    int64_t xs, ys;   // elements from token to token
    int heads;
};

struct RopeParams {
    RopeSide q, k;
    const int32_t *pos;
    const uint64_t *table;
    int64_t n_tokens;
    int dim, rot, per_block;
    float amplitude;
    bool inverse;
    int turn_units, units;   // threads of a head: turning, turning + copying
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

template <typename T, int N>
struct alignas(N * sizeof(T)) Pack {
    T v[N];
};

// Element i of the pair and its partner, turned (cs = amplitude cos, amplitude sin).
template <typename T>
__device__ __forceinline__ void turn(T &a, T &b, float2 cs) {
    const float x = to_f(a), y = to_f(b);
    a = from_f<T>(x * cs.x - y * cs.y);
    b = from_f<T>(x * cs.y + y * cs.x);
}

// N elements per thread and access: 16 bytes where sizes, strides and
// alignment allow, else 1.  threadIdx.x walks the units of one head,
// threadIdx.y the (token, head) rows.
template <typename T, int N, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeParams p) {
    __shared__ float2 cs[kRopePairs];
    let_next_start();
    wait_for_inputs();
    const int pairs = p.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * p.per_block;
    const int nt = (int)min((int64_t)p.per_block, p.n_tokens - t0);
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
    for (int i = tid; i < nt * pairs; i += nthr) {
        const int t = i / pairs, j = i - t * pairs;
        const uint64_t turns = (uint64_t)(int64_t)p.pos[t0 + t] * p.table[j];
        // the nearest quarter turn comes off as an integer: what fp32 then rounds
        // is an eighth of a turn at most
        const uint64_t quarter = (turns + (1ull << 61)) >> 62;
        float s, c;
        sincospif((float)(int64_t)(turns - (quarter << 62)) * 0x1p-63f, &s, &c);
        if (quarter & 1) {
            const float x = c;
            c = -s;
            s = x;
        }
        if (quarter & 2) {
            c = -c;
            s = -s;
        }
        cs[i] = make_float2(p.amplitude * c, p.amplitude * (p.inverse ? -s : s));
    }
    __syncthreads();
    const int unit = threadIdx.x;
    const int heads = p.q.heads + p.k.heads;
    for (int row = threadIdx.y; row < nt * heads; row += blockDim.y) {
        const int t = row / heads, h = row - t * heads;
        const bool is_k = h >= p.q.heads;
        const RopeSide &side = is_k ? p.k : p.q;
        const int64_t at = (int64_t)(is_k ? h - p.q.heads : h) * p.dim;
        const T *x = static_cast<const T *>(side.x) + (t0 + t) * side.xs + at;
        T *y = static_cast<T *>(side.y) + (t0 + t) * side.ys + at;
        const float2 *c = cs + t * pairs;
        using P = Pack<T, N>;
        if (unit >= p.turn_units) {   // behind the turned part
            const int i = p.rot + (unit - p.turn_units) * N;
            *reinterpret_cast<P *>(y + i) = *reinterpret_cast<const P *>(x + i);
        } else if constexpr (INTER) {
            constexpr int M = N < 2 ? 2 : N;   // whole pairs
            alignas(16) T v[M];
            const int i = unit * M;
#pragma unroll
            for (int j = 0; j < M; j += N)
                *reinterpret_cast<P *>(v + j) = *reinterpret_cast<const P *>(x + i + j);
#pragma unroll
            for (int j = 0; j < M; j += 2) turn(v[j], v[j + 1], c[(i + j) / 2]);
#pragma unroll
            for (int j = 0; j < M; j += N)
                *reinterpret_cast<P *>(y + i + j) = *reinterpret_cast<const P *>(v + j);
        } else {
            const int i = unit * N;
            P a = *reinterpret_cast<const P *>(x + i);
            P b = *reinterpret_cast<const P *>(x + i + pairs);
#pragma unroll
            for (int j = 0; j < N; ++j) turn(a.v[j], b.v[j], c[i + j]);
            *reinterpret_cast<P *>(y + i) = a;
            *reinterpret_cast<P *>(y + i + pairs) = b;
        }
    }
}

template <typename T, int N, bool INTER>
void launch(RopeParams &p, bool in_place, int sms, cudaStream_t st) {
    p.turn_units = INTER ? p.rot / (N < 2 ? 2 : N) : p.rot / 2 / N;
    p.units = p.turn_units + (in_place ? 0 : (p.dim - p.rot) / N);
    // tokens of a block: enough blocks for four per SM before angles are
    // shared by more rows, and never more angles than the array holds
    const int64_t want = (p.n_tokens + 4 * sms - 1) / (4 * sms);
    p.per_block = (int)std::min<int64_t>({std::max<int64_t>(1, want), kRopePairs / (p.rot / 2), 8});
    const dim3 block(p.units, std::max(1, kRopeThreads / p.units));
    launch_early(rope_kernel<T, N, INTER>, (unsigned)((p.n_tokens + p.per_block - 1) / p.per_block), block, 0,
                 st, p);
}

template <typename T>
void launch_type(RopeParams &p, bool inter, bool in_place, bool wide, int sms, cudaStream_t st) {
    constexpr int N = 16 / sizeof(T);
    if (wide)
        inter ? launch<T, N, true>(p, in_place, sms, st) : launch<T, N, false>(p, in_place, sms, st);
    else
        inter ? launch<T, 1, true>(p, in_place, sms, st) : launch<T, 1, false>(p, in_place, sms, st);
}

}  // namespace

int launch_rope_table(int32_t rot, double theta, double factor, double alpha, double beta,
                      double context, uint64_t *table, cudaStream_t st) {
    rope_table_kernel<<<(rot / 2 + kTableThreads - 1) / kTableThreads, kTableThreads, 0, st>>>(rot, theta, factor, alpha, beta, context, table);
    return cache_launched("kvc_rope_table");
}

int launch_rope(const RopeArgs &a, int sms, cudaStream_t st) {
    RopeParams p;
    p.q = {a.q, a.q_out, a.q_stride, a.q_out_stride, a.n_q_heads};
    p.k = {a.k, a.k_out, a.k_stride, a.k_out_stride, a.n_k_heads};
    p.pos = a.positions;
    p.table = a.table;
    p.n_tokens = a.n_tokens;
    p.dim = a.head_dim;
    p.rot = a.rot_dim;
    p.amplitude = a.amplitude;
    p.inverse = a.flags & KVC_ROPE_INVERSE;
    const bool inter = a.flags & KVC_ROPE_INTERLEAVED;
    const bool in_place = (a.n_q_heads == 0 || a.q == a.q_out) && (a.n_k_heads == 0 || a.k == a.k_out);
    const int n = a.dtype == KVC_F32 ? 4 : 8;
    // 16-byte accesses: every head, half and tail starts on a boundary
    bool wide = a.head_dim % n == 0 && a.rot_dim % n == 0 && (inter || (a.rot_dim / 2) % n == 0);
    const RopeSide *sides[2] = {&p.q, &p.k};
    for (const RopeSide *s : sides)
        if (s->heads)
            wide = wide && ((reinterpret_cast<uintptr_t>(s->x) | reinterpret_cast<uintptr_t>(s->y)) & 15) == 0 &&
                   s->xs % n == 0 && s->ys % n == 0;
    if (a.dtype == KVC_F32)
        launch_type<float>(p, inter, in_place, wide, sms, st);
    else
        launch_type<__nv_bfloat16>(p, inter, in_place, wide, sms, st);
    return cache_launched("kvc_rope");
}

}  // namespace kvc
