// quant.cuh -- rows held in 4 or 8 bits: the format, and where a row's parts lie.
//
// A row of K or V is cut into groups of 32 channels, the last one filled up with
// zeros.  A group x has codes n of b bits, a step s and a zero code z; it stands
// for (n - z) s.  With N = 2^b - 1 and fl() the rounding to fp32:
//   lo = min(0, min x), hi = max(0, max x)
//   s  = fl((hi/2 - lo/2) / (N/2)) rounded up to four significant bits (b = 4)
//        or to a power of two (b = 8), 2^-126 at least
//   z  = rint(fl(-lo fl(1/s))),  n = min(max(rint(fl(x fl(1/s))) + z, 0), N)
// Steps of so few bits make (n - z) s exact in bf16: |n - z| <= N has b bits, s
// the other four or one.  They are up to an eighth (b = 4) or twice (b = 8) as
// wide as they need be.  A zero code of its own, and not the middle one, because
// a group's values often lie to one side (a strong channel of K is one of its 32).
// A group with a value not below 2^126 in size -- an infinity, a NaN -- stands
// for NaN.
//
// s and z take 16 bits: b = 4, s as bf16 with z in its four lowest bits; b = 8, the
// exponent of s (biased by 127) above z.  A step that is NaN or infinite marks a
// group that stands for NaN: its codes and z are zero, and zero times either is NaN.
//
// Pools are made of blocks of 16 rows: the rows' codes, then their groups' words.  A
// block is one stretch of memory, whatever the page size, so any 16 rows of a page
// come with one bulk copy.  A row's codes are ordered for the fragments of the
// warp-wide matrix instruction that reads them (attend_quant.cu), in pieces of
// eight channels, piece c of group g: the codes of K as word c G + g (b = 4; of a
// row of G groups) or words 2 (c G + g), .. + 1 (b = 8), so that a lane that owns
// column c finds all its groups in a row; those of V as two halves, 2 c and 2 c + 1,
// half h of group g as 16-bit (b = 4) or 32-bit (b = 8) word h G + g.  In a piece
// of 4-bit codes channel 2 i is nibble i, channel 2 i + 1 nibble i + 4; V's halves
// are the even and the odd channels.  8-bit codes are in channel order.
#pragma once

#include "cache.cuh"

namespace kvc {

constexpr int kQuantRows = 16;   // rows of a block
constexpr int kQuantGroup = 32;  // channels of a group

__host__ __device__ constexpr int quant_groups(int dim) { return (dim + kQuantGroup - 1) / kQuantGroup; }
// Bytes of a row's codes, of its groups' words, and of a block.
__host__ __device__ constexpr int quant_codes(int bits, int groups) { return 4 * bits * groups; }
__host__ __device__ constexpr int quant_words(int groups) { return 2 * groups; }
__host__ __device__ constexpr int quant_block(int bits, int groups) {
    return kQuantRows * (quant_codes(bits, groups) + quant_words(groups));
}

// Where row `row` (counted over the whole pool) of a pool has its codes and words.
struct QuantRow {
    int64_t codes, words;   // bytes from the pool's beginning
};
__device__ __forceinline__ QuantRow quant_row(int bits, int groups, int64_t row) {
    const int64_t block = (row >> 4) * quant_block(bits, groups);
    const int i = (int)(row & 15);
    return {block + i * quant_codes(bits, groups),
            block + kQuantRows * quant_codes(bits, groups) + i * quant_words(groups)};
}

// The step and zero code of a group's word.
template <int BITS>
__device__ __forceinline__ float quant_step(uint32_t word) {
    return BITS == 4 ? __uint_as_float((word & 0xfff0u) << 16) : __uint_as_float((word & 0xff00u) << 15);
}
template <int BITS>
__device__ __forceinline__ int quant_zero(uint32_t word) {
    return word & (BITS == 4 ? 0xfu : 0xffu);
}
// Whether a group stands for NaN.
template <int BITS>
__device__ __forceinline__ bool quant_is_nan(uint32_t word) {
    constexpr uint32_t kExponent = BITS == 4 ? 0x7f80u : 0xff00u;
    return (word & kExponent) == kExponent;
}

// A piece's codes as they are computed: 4 bits, the word of the comment above in
// .x; 8 bits, channels 0-3 in .x and 4-7 in .y.
template <int BITS>
__device__ __forceinline__ uint2 quant_load(const uint8_t *codes, int groups, int g, int c, bool of_v) {
    const int at = c * groups + g;
    if (BITS == 8) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(codes);
        if (!of_v) return *reinterpret_cast<const uint2 *>(p + 2 * at);
        return make_uint2(p[at + c * groups], p[at + (c + 1) * groups]);
    }
    if (!of_v) return make_uint2(reinterpret_cast<const uint32_t *>(codes)[at], 0);
    const uint16_t *p = reinterpret_cast<const uint16_t *>(codes);
    return make_uint2(p[at + c * groups] | (uint32_t)p[at + (c + 1) * groups] << 16, 0);
}
template <int BITS>
__device__ __forceinline__ void quant_store(uint8_t *codes, int groups, int g, int c, bool of_v, uint2 x) {
    const int at = c * groups + g;
    if (BITS == 8) {
        uint32_t *p = reinterpret_cast<uint32_t *>(codes);
        if (!of_v) {
            *reinterpret_cast<uint2 *>(p + 2 * at) = x;
        } else {
            p[at + c * groups] = x.x;
            p[at + (c + 1) * groups] = x.y;
        }
    } else if (!of_v) {
        reinterpret_cast<uint32_t *>(codes)[at] = x.x;
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(codes);
        p[at + c * groups] = (uint16_t)x.x;
        p[at + (c + 1) * groups] = (uint16_t)(x.x >> 16);
    }
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What a piece stands for, as bf16, which holds it exactly; `word` is the group's,
// once in either half.  Codes come as 128 + n (4 bits), where bf16 counts in ones, or
// as 2^23 + n in fp32 (8 bits); the zero code comes off the same way.
template <int BITS>
__device__ __forceinline__ void quant_bf16(uint2 codes, uint32_t word, uint32_t (&y)[4]) {
    if (BITS == 4) {
        const uint32_t s = word & 0xfff0fff0u, z = (word & 0x000f000fu) | 0x43004300u;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul_bf16x2(sub_bf16x2(((codes.x >> 4 * i) & 0x000f000fu) | 0x43004300u, z), s);
    } else {
        const float s = quant_step<8>(word), z = -__uint_as_float(0x4b000000u | (word & 0xffu));
        const unsigned long long s2 = f2_pack(s, s), z2 = f2_pack(z, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = i < 2 ? codes.x : codes.y;
            float a, b;
            f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + 2 * (i & 1))),
                                            __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + 2 * (i & 1)))), z2), s2), a, b);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[i]) : "f"(b), "f"(a));
        }
    }
}

// The smallest and largest of eight channels and zero; NaN and infinities make the
// largest infinite.
__device__ __forceinline__ void quant_range(const float (&x)[8], float *lo, float *hi) {
    *lo = fminf(fmin3(fminf(fmin3(x[0], x[1], x[2]), fmin3(x[3], x[4], x[5])), x[6], x[7]), 0.f);
    *hi = fmaxf(fmax3(fmaxf(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5])), x[6], x[7]), 0.f);
    unsigned long long odd = 0;   // stays zero but for those
#pragma unroll
    for (int i = 0; i < 8; i += 2) odd = f2_fma(f2_pack(x[i], x[i + 1]), f2_pack(0.f, 0.f), odd);
    float a, b;
    f2_unpack(odd, a, b);
    if (!(a + b == 0.f)) *hi = INFINITY;
}

// Codes of eight channels, by 1 / s and z: rounding by adding 1.5 2^23, where fp32
// counts in ones (conversions run at an eighth of the rate).  rint(x / s) + z is never
// below 0: lo has the smallest, and -z exactly.
template <int BITS>
__device__ __forceinline__ uint2 quant_codes_of(const float (&x)[8], float inv, float z) {
    constexpr float kOnes = 12582912.f, kMost = kOnes + (1 << BITS) - 1;
    const unsigned long long z2 = f2_pack(z, z);
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        // the product is rounded before the sum (a packed product and sum would be fused)
        const float p = __fadd_rn(__fmul_rn(x[i], inv), kOnes), q = __fadd_rn(__fmul_rn(x[i + 1], inv), kOnes);
        float a, b;
        f2_unpack(f2_add(f2_pack(p, q), z2), a, b);
        n[i] = __float_as_uint(fminf(a, kMost));
        n[i + 1] = __float_as_uint(fminf(b, kMost));
    }
    if (BITS == 8)
        return make_uint2(__byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410));
    uint32_t r = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) r = r * 16 + __byte_perm(n[2 * i], n[2 * i + 1], 0x5410);
    return make_uint2(r, 0);
}

// Codes and words of a group of K and one of V from their values, eight in each of four
// neighbouring lanes; the lanes of `mask` call it together.  Even lanes work K's step
// out, odd ones V's.
template <int BITS>
__device__ __forceinline__ void quant_encode(const float (&kx)[8], const float (&vx)[8], uint32_t mask, uint2 *kc, uint32_t *kw, uint2 *vc,
                                             uint32_t *vw) {
    constexpr int N = (1 << BITS) - 1;
    constexpr float kOnes = 12582912.f;
    float klo, khi, vlo, vhi;
    quant_range(kx, &klo, &khi);
    quant_range(vx, &vlo, &vhi);
    // lane c gets the range of its own of the two over lanes c and c ^ 1, then over all
    const int lane = threadIdx.x & 31, odd = lane & 1;
    float lo = odd ? vlo : klo, hi = odd ? vhi : khi;
    lo = fminf(lo, __shfl_xor_sync(mask, odd ? klo : vlo, 1));
    hi = fmaxf(hi, __shfl_xor_sync(mask, odd ? khi : vhi, 1));
    lo = fminf(lo, __shfl_xor_sync(mask, lo, 2));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, 2));
    const bool fine = fmaxf(-lo, hi) < 0x1p126f;
    const float t = __fdiv_rn(__fadd_rn(hi * 0.5f, lo * -0.5f), 0.5f * N);
    constexpr uint32_t kDropped = BITS == 4 ? 20 : 23;   // bits of fp32 that are rounded up
    uint32_t s_bits = (__float_as_uint(t) + ((1u << kDropped) - 1u)) >> kDropped << kDropped;
    s_bits = max(s_bits, __float_as_uint(0x1p-126f));
    const float inv = __frcp_rn(__uint_as_float(s_bits)), z = __fadd_rn(__fmul_rn(-lo, inv), kOnes);
    const uint32_t z_bits = __float_as_uint(z) & 0xffu;
    const uint32_t word = !fine ? (BITS == 4 ? 0x7fc0u : 0xff00u) : BITS == 4 ? s_bits >> 16 | z_bits : s_bits >> 23 << 8 | z_bits;
    const int even = lane & ~1;
    *kw = __shfl_sync(mask, word, even);
    *vw = __shfl_sync(mask, word, even + 1);
    const float k_inv = __shfl_sync(mask, inv, even), v_inv = __shfl_sync(mask, inv, even + 1);
    constexpr uint32_t kZero = BITS == 4 ? 0xfu : 0xffu;
    *kc = quant_codes_of<BITS>(kx, k_inv, __uint_as_float(__float_as_uint(kOnes) | (*kw & kZero)) - kOnes);
    *vc = quant_codes_of<BITS>(vx, v_inv, __uint_as_float(__float_as_uint(kOnes) | (*vw & kZero)) - kOnes);
    if (quant_is_nan<BITS>(*kw)) *kc = make_uint2(0, 0);
    if (quant_is_nan<BITS>(*vw)) *vc = make_uint2(0, 0);
}

int launch_pages_append_quant(const kvc_cache &c, int bits, const PagesState &s, int32_t *table, int32_t *len,
                              int32_t n_lists, const int32_t *counts, const int64_t *src_row, int64_t src_step,
                              const void *k_src, const void *v_src, int64_t src_rows, void *k_pool, void *v_pool,
                              int sms, cudaStream_t st);
int launch_pages_compact_quant(const kvc_cache &c, int bits, const PagesState &s, int32_t *table, int32_t *len,
                               int32_t n_lists, const int32_t *idx, int32_t k_max, const int32_t *counts,
                               void *k_pool, void *v_pool, int sms, cudaStream_t st);
int launch_pages_read_quant(const kvc_cache &c, int bits, const PagesState &s, const int32_t *table,
                            const int32_t *len, int32_t n_lists, const int32_t *first, const int32_t *counts,
                            const int64_t *dst_row, int64_t dst_step, const void *k_pool, const void *v_pool,
                            void *k_dst, void *v_dst, int64_t dst_rows, int sms, cudaStream_t st);

}  // namespace kvc
