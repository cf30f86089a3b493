// attend_quant.cu -- attention of few rows over a cache held in 4 or 8 bits: bf16
// queries of head size 64 or 128, units of up to 8 NT rows (tokens x the KV head's query
// heads) of a list, up to 32 rows in all.  What a decode step or a draft is made of;
// longer lists of rows are attend_tc.cuh's.
//
// Reading the cache should bound it: a code may then cost three instructions, so none
// is spent on taking it out of the packed word but the one that picks it.  With codes n,
// step s and zero code z of a key's group, and everything per row (query head) of the list:
//   logit  = sum_g s_g (sum_d q_d n_d - z_g sum_d q_d)
//   out_d  = sum_t (p_t s_tg) (n_td - z_tg)
// The sums are matrix products (mma.m16n8k16).  K's is with the codes as they are: a code
// picked out of its word by a mask is an fp16 number as it stands, n 2^-24 in bits 0-3 (or
// 0-7) of a half and n 2^-20 in bits 4-7, exactly; the rows of Q that meet the latter are
// 2^4 apart, and the groups' steps and zero codes go to the products' 16 x 8 results in fp32.
//
// V's is in bf16, whose exponents are fp32's, so that no value is too large or too small
// beside another one: a code as it stands is n 2^-133 or n 2^-129 there, and one
// multiplication and sum makes it (n - z) 2^-20, exactly; a value of 0 is 0 in the product.
// What a row's probability times the group's step is rounded to is two bf16 numbers,
// 2^-17 of it away at most, as the tensor cores' other kernels have it.  (One fp16 number
// instead, steps over the list's largest and the zero codes' share in a product of its own:
// 7-9% less time, but 7 to 17% of the outputs were not the nearest number, and what one row
// held far above the others, seen or not, took their bits.)
//
// Fragments: the product of K has 16 keys as its rows and 8 of the list's rows as
// columns, a step of 16 channels picks two codes per lane out of every key's word, in
// the order that quant.cuh lays down, so a lane loads all its codes of a key at once.
// Its result, turned by movmatrix, is the second operand of V's product, whose rows
// are channels.  Key i of a block stands in row pi(i) of both products: pi(2 c) = c,
// pi(2 c + 1) = 4 + (c ^ 1), for fewer bank conflicts.
//
// P: 2^24 for a probability of 1 (the running maximum may lag behind by 2^4), so that
// rows whose values are near the type's smallest keep the bits of small probabilities; with
// the values' 2^-20 the sums stand 2^4 above the outputs, and values of 2^100 fit them.
//
// Every warp walks 32 keys of each step of 128 by itself, with a ring of its own that
// bulk copies fill (a block of K or V of 16 rows each); the warps' results meet in
// shared memory at the end of a list.  Work is split as in attend.cuh.
//
// What bounds it, measured on one GB300 (measured copy rate 6,776 GB/s):
// - 8 bits: reading the cache, once lists are long.  32 sequences x 8 KV heads over
//   4,000-48,000 rows: 315 us, 5.7 TB/s, 85%; over 500-6,000: 57-58 us, 3.9 TB/s, the rest
//   of which is about 20 us of plan (7), first loads (6) and joining at lists' ends.
// - 4 bits: instructions and the latency between them.  About 950 per 32 keys, warp and 128
//   channels would take 44 us of issue for 64 x 8 lists of 500-6,000 rows; the twelve warps
//   that an SM holds issue at half that rate: 82 us, 2.9 TB/s, 43%; of 4,000-48,000: 510
//   us, 3.8 TB/s.
// - 17 to 32 rows: the same with 8 warps to an SM, for the registers.  3 x 4 lists of
//   60,000-131,000 rows, 28 rows, heads of 64: 84-86 us.
// - one sequence of 1,000 rows: latency, 11-12 us.
#include <climits>

#include "attend.cuh"
#include "quant.cuh"

namespace kvc {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kChunk = 32;                 // keys of a warp's step
constexpr int kStepKeys = kWarps * kChunk;
constexpr int kSlotRows = 32;
// Blocks per SM by their registers: 128, 168 or 255 per thread.  A head of 64 spills
// less than its one block more gains (64 x 8 lists of 500-6,000 rows in 4 bits: 16 rows 79
// us with three, 85 with two; 8 rows 58 with four, 60 with three).  One of 128 does not (16
// rows: 136 us with three, 120 with two; in 8 bits, 32 x 8 lists, 97 and 75; 8 rows: 91
// with four, 82 with three, 90 with two; in 8 bits 70, 58 and 62).
constexpr int per_sm_of(int groups, int nt) {
    return groups == 2 ? (nt == 1 ? 4 : nt == 2 ? 3 : 2) : nt == 1 ? 3 : 2;
}
// A unit costs about two steps beside its steps (us with 0, 2, 4 and 6: 64 x 8 lists of
// 500-6,000 rows in 4 bits 83.4, 82.3, 84.1, 87.3; 32 x 8 in 8 bits 61.0, 58.9, 60.3,
// 62.9; 12 lists of 60,000-131,000 88.3, 83.6, 82.9, 82.9).
constexpr int kExtra = 2;
constexpr float kLag = 4.f;                // log2 units m may lag behind
constexpr float kTop = 24.f;               // log2 of what P has for a probability of 1

// Ring slots of a warp.
constexpr int slots_of(int bits, int groups) { return bits == 4 && groups == 2 ? 4 : 2; }
constexpr int slot_bytes(int bits, int groups) { return 4 * quant_block(bits, groups); }   // K K V V
// K's steps and zero codes in fp32, V's in bf16.
constexpr int scratch_bytes(int groups) { return kChunk * groups * 8 + 2 * kChunk / 2 * groups * 4; }
constexpr int out_floats(int groups) { return kWarps * 8 * (32 * groups + 1); }
constexpr int ring_bytes(int bits, int groups) {
    const int ring = kWarps * slots_of(bits, groups) * slot_bytes(bits, groups), out = out_floats(groups) * 4;
    return ring > out ? ring : (out + 15) / 16 * 16;
}

template <int SLOTS>
struct Shared {
    uint64_t full[kWarps][SLOTS];
    float2 stat[kWarps][8];
    int64_t plan[kWarps + 4];
    int stop;
    uint32_t last;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The transpose of an 8 x 8 matrix of 16-bit elements, a pair of a row per lane.
__device__ __forceinline__ uint32_t turn(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// What (hi + lo) s has beside `product`, the rounded hi s: with 8 bits s is a power of two
// and hi s is exact.
template <int BITS>
__device__ __forceinline__ uint32_t rest_of(uint32_t hi, uint32_t lo, uint32_t s, uint32_t product) {
    if (BITS == 8) return mul_bf16x2(lo, s);
    return fma_bf16x2(lo, s, fma_bf16x2(hi, s, product ^ 0x80008000u));
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x) {
    float2 r;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(x));
    return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // -127 .. 127

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The four pairs of codes of a piece of K (4 bits: of one word, 8 bits: of two), each
// a pair of fp16 numbers; those of odd places 2^4 as large with 4 bits.
template <int BITS>
__device__ __forceinline__ void pick(uint32_t w0, uint32_t w1, uint32_t (&e)[4]) {
    if (BITS == 4) {
        const uint32_t up = w0 >> 8;
        e[0] = w0 & 0x000f000fu;
        e[1] = w0 & 0x00f000f0u;
        e[2] = up & 0x000f000fu;
        e[3] = up & 0x00f000f0u;
    } else {
        e[0] = w0 & 0x00ff00ffu;
        e[1] = w0 >> 8 & 0x00ff00ffu;
        e[2] = w1 & 0x00ff00ffu;
        e[3] = w1 >> 8 & 0x00ff00ffu;
    }
}

// Of a list's row r: channels 32 g + 8 c .. + 7.
__device__ __forceinline__ uint4 load_q(const AttendParams &p, const AttendUnit &a, int r, int g, int c) {
    if (r >= a.rows) return make_uint4(0, 0, 0, 0);
    const int token = p.by_group(a.row0 + r);
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (a.q0 + token) * p.q_stride +
                             (int64_t)(a.h * p.group + a.row0 + r - token * p.group) * p.dim + 32 * g + 8 * c;
    return *reinterpret_cast<const uint4 *>(q);
}

template <int G, int BITS, int NT>
__global__ void __launch_bounds__(kThreads, per_sm_of(G, NT)) attend_quant_kernel(const __grid_constant__ AttendParams p) {
    constexpr int D = 32 * G, kSlots = slots_of(BITS, G), kBlock = quant_block(BITS, G), kCodes = quant_codes(BITS, G);
    constexpr int kRow = kCodes, kWordsAt = kQuantRows * kCodes, kOutRow = D + 1;
    extern __shared__ __align__(128) uint8_t raw[];
    uint8_t *ring = raw;
    float *s_out = reinterpret_cast<float *>(raw);   // the warps' results, when the ring is at rest
    uint8_t *scratch_all = raw + ring_bytes(BITS, G);
    Shared<kSlots> &s = *reinterpret_cast<Shared<kSlots> *>(scratch_all + kWarps * scratch_bytes(G));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c = lane & 3;
    uint8_t *mine = ring + warp * kSlots * slot_bytes(BITS, G);
    float2 *k_steps = reinterpret_cast<float2 *>(scratch_all + warp * scratch_bytes(G));   // [key][G]: s, -s z
    uint32_t *steps = reinterpret_cast<uint32_t *>(k_steps + kChunk * G);                    // V: [pair of keys][G]
    uint32_t *zeros = steps + kChunk / 2 * G;                                                // the same of -z 2^-20
    volatile int *stop = &s.stop;
    const int key_of[2] = {(r8 & 1) ? 4 + (r8 >> 1 ^ 1) : r8 >> 1, 8 + ((r8 & 1) ? 4 + (r8 >> 1 ^ 1) : r8 >> 1)};   // of rows r8, r8 + 8
    // the lane's own key of the 32, and its half of its pair's word
    const int my_k = lane & 7, my_pair = (lane >> 3) * 4 + (my_k < 4 ? my_k : (my_k - 4) ^ 1), my_half = my_k >= 4;

    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < kSlots; ++i) mbar_init(&s.full[w][i], 1);
        s.stop = 0;
        fence_barrier_init();
    }
    let_next_start();
    wait_for_inputs();
    const AttendRun run = attend_plan<kThreads, true>(p, s.plan);   // (its barrier is the barriers' too)
    if (run.lo >= run.hi) return;
    uint32_t slot = 0, round = 0;   // the slot that is next, and how often it has been
    uint32_t pending = 0, first_ask = 1;
    bool ok = true;
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
        // ---------------------------------------------------- loads
        const int32_t *entry = p.table + (int64_t)a.list * p.max_pages;
        // page numbers of the warp's blocks, 16 steps at a time
        auto look_up = [&](int batch) {
            const int64_t key = (int64_t)(t0 + batch * 16 + (lane >> 1)) * kStepKeys + warp * kChunk + kQuantRows * (lane & 1);
            return key < a.hi ? entry[key >> p.shift] : 0;
        };
        int batch = 0, now = look_up(0), then = look_up(1), next = t0;
        uint32_t absent = 0;   // two bits per slot: blocks that are not there
        // the warp's blocks of step `next` into slot `to`
        auto ask = [&](uint32_t to) {
            const int at = 2 * (next - t0);
            if (at >> 5 > batch) {
                ++batch;
                now = then;
                then = look_up(batch + 1);
            }
            const int key = next * kStepKeys + warp * kChunk;   // (its blocks may lie past a.hi)
            const int page0 = __shfl_sync(0xffffffffu, now, at & 31), page1 = __shfl_sync(0xffffffffu, now, (at + 1) & 31);
            const bool seen0 = key < a.hi, seen1 = key + kQuantRows < a.hi;
            const bool there0 = seen0 && (uint32_t)page0 < (uint32_t)p.n_pages, there1 = seen1 && (uint32_t)page1 < (uint32_t)p.n_pages;
            absent = (absent & ~(3u << 2 * to)) | (uint32_t)(!there0 | !there1 << 1) << 2 * to;
            if (lane == 0) {
                if ((seen0 && !there0) || (seen1 && !there1)) set_status(p.status, KVC_DEV_BAD_PAGE);
                if (!(p.skip_load && first_ask)) {
                    uint64_t *bar = &s.full[warp][to];
                    const uint32_t bytes = (there0 + there1) * 2 * kBlock;
                    if (bytes)
                        mbar_arrive_expect_tx(bar, bytes);
                    else
                        mbar_arrive(bar);
                    uint8_t *dst = mine + to * slot_bytes(BITS, G);
                    const int in_page = (key & ((1 << p.shift) - 1)) >> 4;
                    if (there0) {
                        const int64_t at0 = ((int64_t)page0 << (p.shift - 4)) + in_page;
                        bulk_load(dst, static_cast<const uint8_t *>(p.k_pool) + at0 * kBlock, kBlock, bar);
                        bulk_load(dst + 2 * kBlock, static_cast<const uint8_t *>(p.v_pool) + at0 * kBlock, kBlock, bar);
                    }
                    if (there1) {   // the next block of the page, or the first of the next page
                        const int64_t at1 = ((int64_t)page1 << (p.shift - 4)) + (p.shift == 4 ? 0 : in_page + 1);
                        bulk_load(dst + kBlock, static_cast<const uint8_t *>(p.k_pool) + at1 * kBlock, kBlock, bar);
                        bulk_load(dst + 3 * kBlock, static_cast<const uint8_t *>(p.v_pool) + at1 * kBlock, kBlock, bar);
                    }
                }
            }
            first_ask = 0;
            ++pending;
            ++next;
        };
        for (uint32_t i = 0, to = slot; ok && i < kSlots && next < t1; ++i, to = to + 1 == kSlots ? 0 : to + 1) ask(to);

        // ---------------------------------------------------- queries
        // of row 8 nt + r8, piece c of every group, as fp16 over a power of two
        uint32_t q[NT][G][4];
        float qs[NT][G][2];   // of the lane's two columns: the group's sum
        float factor[NT][2];  // logit in log2 units of a sum
        int sees[NT][2];
        float mul[NT];        // the lane's row's
        bool far = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint4 x[G];
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                x[g] = load_q(p, a, 8 * nt + r8, g, c);
                const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max(top, max(w[i] << 16 & 0x7fffffffu, w[i] & 0x7fff0000u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int f = min(10 + 127 - (int)(top >> 23), 126);   // the largest becomes 2^10 and more
            const float up = pow2(f);
            float sum[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
                float y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[2 * i] = __uint_as_float(w[i] << 16) * up;
                    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * up;
                }
                sum[g] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the pairs that pick() makes; 2^4 more where the code is at 2^-24
                    const int i0 = BITS == 4 ? 2 * i : 4 * (i >> 1) + (i & 1), i1 = BITS == 4 ? i0 + 1 : i0 + 2;
                    const float more = BITS == 8 || i % 2 == 0 ? 16.f : 1.f;
                    q[nt][g][i] = pack_f16(y[i0] * more, y[i1] * more);
                    const float2 z = unpack_f16(q[nt][g][i]);
                    sum[g] += (z.x + z.y) * (1.f / more);
                }
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
            }
            mul[nt] = p.scale_log2 * pow2(-f);
            far |= !isfinite(mul[nt] * 0x1p20f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * c + e) * 4, row = 8 * nt + 2 * c + e;
#pragma unroll
                for (int g = 0; g < G; ++g) qs[nt][g][e] = __shfl_sync(0xffffffffu, sum[g], from) * 0x1p-20f;
                sees[nt][e] = row < a.rows ? attend_sees(p, a, row) : 0;
            }
        }
        // codes times q are at 2^-20, which the factor takes back; that of queries of 2^120
        // would not be a number, so logits and m stay 2^-20 of what they are until the exponentials
        const float up = __any_sync(0xffffffffu, far) ? 0x1p20f : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                factor[nt][e] = __shfl_sync(0xffffffffu, mul[nt] * (up == 1.f ? 0x1p20f : 1.f), (2 * c + e) * 4);
        const int sees0 = attend_sees(p, a, 0);   // the fewest

        float m[NT][2], l[NT][2], o[NT][2 * G][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int mt = 0; mt < 2 * G; ++mt) o[nt][mt][i] = 0.f;
            }
        }

        for (int t = t0; ok && t < t1; ++t) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s.full[warp][slot], round & 1, stop, p.status));
            if (!ok) break;
            --pending;
            const uint8_t *k_at = mine + slot * slot_bytes(BITS, G), *v_at = k_at + 2 * kBlock;
            const int key0 = t * kStepKeys + warp * kChunk;
            const uint32_t gone = absent >> 2 * slot & 3;
            // ------------------------------------------------ steps and zero codes, a key per lane
            bool odd = false;
            {
                const bool there = key0 + lane < a.hi && !(gone >> (lane >> 4) & 1);
                const uint32_t is = there ? 0xffffffffu : 0;   // (a row that is not there has steps of zero)
                const int at = (lane >> 4) * kBlock + kWordsAt + (lane & 15) * quant_words(G);
                uint32_t kw[G / 2], vw[G / 2];
                if (G == 4) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(k_at + at), z = *reinterpret_cast<const uint2 *>(v_at + at);
                    kw[0] = y.x & is;
                    kw[G / 2 - 1] = y.y & is;
                    vw[0] = z.x & is;
                    vw[G / 2 - 1] = z.y & is;
                } else {
                    kw[0] = *reinterpret_cast<const uint32_t *>(k_at + at) & is;
                    vw[0] = *reinterpret_cast<const uint32_t *>(v_at + at) & is;
                }
                uint32_t nan = 0;
#pragma unroll
                for (int i = 0; i < G / 2; ++i) {
                    // V's steps are bf16 numbers
                    uint32_t vs = BITS == 4 ? vw[i] & 0xfff0fff0u : vw[i] >> 1 & 0x7f807f80u;
                    const uint32_t none = (vs & 0x7f807f80u) + 0x00800080u & 0x80008000u;   // exponents of ones only
                    nan |= none;
                    vs &= ~((none >> 15) * 0xffffu);   // added below
                    // -z 2^-20: a whole number below 256 is that number times 2^-133 as bf16
                    const uint32_t vz = mul_bf16x2(vw[i] & (BITS == 4 ? 0x000f000fu : 0x00ff00ffu), 0xf800f800u);
                    uint16_t *s16 = reinterpret_cast<uint16_t *>(steps) + (my_pair * G + 2 * i) * 2 + my_half;
                    uint16_t *z16 = reinterpret_cast<uint16_t *>(zeros) + (my_pair * G + 2 * i) * 2 + my_half;
                    s16[0] = (uint16_t)vs;
                    s16[2] = (uint16_t)(vs >> 16);
                    z16[0] = (uint16_t)vz;
                    z16[2] = (uint16_t)(vz >> 16);
                    // zero codes as 1 + z / 16 or 1 + z / 256, for want of a cheap conversion
                    const float s0 = quant_step<BITS>(kw[i] & 0xffffu), s1 = quant_step<BITS>(kw[i] >> 16);
                    float z0, z1;
                    if (BITS == 4) {
                        z0 = fmaf(__uint_as_float((kw[i] << 19 & 0x00780000u) | 0x3f800000u), -16.f, 16.f);
                        z1 = fmaf(__uint_as_float((kw[i] << 3 & 0x00780000u) | 0x3f800000u), -16.f, 16.f);
                    } else {
                        z0 = fmaf(__uint_as_float((kw[i] << 15 & 0x007f8000u) | 0x3f800000u), -256.f, 256.f);
                        z1 = fmaf(__uint_as_float((kw[i] >> 1 & 0x007f8000u) | 0x3f800000u), -256.f, 256.f);
                    }
                    *reinterpret_cast<float4 *>(k_steps + lane * G + 2 * i) = make_float4(s0, s0 * z0, s1, s1 * z1);
                }
                odd = __any_sync(0xffffffffu, nan != 0);   // groups of V that stand for NaN
                __syncwarp();
            }
            // ------------------------------------------------ logits
            float x[2][NT][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t code[2][kCodes / 16];
                float4 st[2][G / 2];   // step and zero code's share, of two groups each
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *at = k_at + b * kBlock + key_of[h] * kRow + c * (kCodes / 4);
                    if (kCodes == 32) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(at);
                        code[h][0] = y.x;
                        code[h][1] = y.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < kCodes / 64; ++i) {
                            const uint4 y = reinterpret_cast<const uint4 *>(at)[i];
                            code[h][4 * i] = y.x;
                            code[h][4 * i + 1] = y.y;
                            code[h][4 * i + 2] = y.z;
                            code[h][4 * i + 3] = y.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < G / 2; ++i)
                        st[h][i] = *reinterpret_cast<const float4 *>(k_steps + (kQuantRows * b + key_of[h]) * G + 2 * i);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[b][nt][i] = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    uint32_t e0[4], e1[4];   // of rows r8 and r8 + 8
                    pick<BITS>(code[0][BITS == 4 ? g : 2 * g], code[0][BITS == 4 ? g : 2 * g + 1], e0);
                    pick<BITS>(code[1][BITS == 4 ? g : 2 * g], code[1][BITS == 4 ? g : 2 * g + 1], e1);
                    const uint32_t a0[4] = {e0[0], e1[0], e0[1], e1[1]}, a1[4] = {e0[2], e1[2], e0[3], e1[3]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        mma16816_zero(d, a0, q[nt][g][0], q[nt][g][1]);
                        mma16816(d, a1, q[nt][g][2], q[nt][g][3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 &w = st[i >> 1][g / 2];
                            x[b][nt][i] = fmaf(g & 1 ? w.w : w.y, qs[nt][g][i & 1], fmaf(g & 1 ? w.z : w.x, d[i], x[b][nt][i]));
                        }
                    }
                }
            }
            // ------------------------------------------------ softmax
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[b][nt][i] *= factor[nt][i & 1];
            if (key0 + kChunk > sees0) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (key0 + kQuantRows * b + key_of[i >> 1] >= sees[nt][i & 1]) x[b][nt][i] = -INFINITY;
            }
            bool grow = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e]));
                    grow |= fmaf(top[nt][e] - m[nt][e], up, -kLag) > 0.f;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = top[nt][e];
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                        y = fmaxf(y, m[nt][e]);
                        const float down = y == -INFINITY ? 1.f : ex2((m[nt][e] - y) * up);
                        m[nt][e] = y;
                        l[nt][e] *= down;
#pragma unroll
                        for (int mt = 0; mt < 2 * G; ++mt) {
                            o[nt][mt][e] *= down;
                            o[nt][mt][2 + e] *= down;
                        }
                    }
            }
            uint32_t pt[2][NT][2], pl[2][NT][2];   // P in two terms, keys the inner dimension: [block][..][keys 0-7, 8-15]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float n0 = m[nt][0] == -INFINITY ? kTop : fmaf(-m[nt][0], up, kTop), n1 = m[nt][1] == -INFINITY ? kTop : fmaf(-m[nt][1], up, kTop);
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ex2(fmaf(x[b][nt][2 * h], up, n0)), p1 = ex2(fmaf(x[b][nt][2 * h + 1], up, n1));
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        const uint32_t hi = pack_bf16(p0, p1);
                        pt[b][nt][h] = turn(hi);
                        pl[b][nt][h] = turn(pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
                    }
            }
            // ------------------------------------------------ values
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // keys that stand at 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the block
                uint32_t code[4][kCodes / 32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = (j & 1 ? 4 + (c ^ 1) : c) + 8 * (j >> 1);
                    const uint8_t *at = v_at + b * kBlock + key * kRow + r8 * (kCodes / 8);
                    if (kCodes == 32) {
                        code[j][0] = *reinterpret_cast<const uint32_t *>(at);
                    } else if (kCodes == 64) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(at);
                        code[j][0] = y.x;
                        code[j][kCodes / 32 - 1] = y.y;
                    } else {
                        const uint4 y = *reinterpret_cast<const uint4 *>(at);
                        code[j][0] = y.x;
                        code[j][1 % (kCodes / 32)] = y.y;
                        code[j][2 % (kCodes / 32)] = y.z;
                        code[j][3 % (kCodes / 32)] = y.w;
                    }
                }
                uint32_t st[2][G], sz[2][G];   // steps and zero codes
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t *at = (h < 2 ? steps : zeros) + (8 * b + 4 * (h & 1) + c) * G;
                    uint32_t(&to)[G] = h < 2 ? st[h & 1] : sz[h & 1];
                    if (G == 4) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(at);
                        to[0] = y.x;
                        to[1] = y.y;
                        to[2 % G] = y.z;
                        to[3 % G] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(at);
                        to[0] = y.x;
                        to[1] = y.y;
                    }
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    // codes of two keys side by side: channels e[0] .. e[3] of the lane's half
                    uint32_t e0[4], e1[4];
                    if (BITS == 4) {
                        const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
                        pick<4>(__byte_perm(code[0][g / 2], code[1][g / 2], sel), 0, e0);
                        pick<4>(__byte_perm(code[2][g / 2], code[3][g / 2], sel), 0, e1);
                    } else {
                        pick<8>(__byte_perm(code[0][g], code[1][g], 0x5410), __byte_perm(code[0][g], code[1][g], 0x7632), e0);
                        pick<8>(__byte_perm(code[2][g], code[3][g], 0x5410), __byte_perm(code[2][g], code[3][g], 0x7632), e1);
                    }
                    // (n - z) 2^-20: as bf16 numbers codes are at 2^-133, those in bits 4-7 at 2^-129
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        constexpr uint32_t kUp = 0x78007800u, kUp4 = 0x76007600u;   // 2^113, 2^109
                        e0[i] = fma_bf16x2(e0[i], BITS == 4 && (i & 1) ? kUp4 : kUp, sz[0][g]);
                        e1[i] = fma_bf16x2(e1[i], BITS == 4 && (i & 1) ? kUp4 : kUp, sz[1][g]);
                    }
                    const uint32_t a0[4] = {e0[0], e0[1], e1[0], e1[1]}, a1[4] = {e0[2], e0[3], e1[2], e1[3]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // p s in two terms: what the first one's rounding leaves is exact
                        const uint32_t b0 = mul_bf16x2(pt[b][nt][0], st[0][g]), b1 = mul_bf16x2(pt[b][nt][1], st[1][g]);
                        const uint32_t c0 = rest_of<BITS>(pt[b][nt][0], pl[b][nt][0], st[0][g], b0);
                        const uint32_t c1 = rest_of<BITS>(pt[b][nt][1], pl[b][nt][1], st[1][g], b1);
                        mma16816_bf16(o[nt][2 * g], a0, b0, b1);
                        mma16816_bf16(o[nt][2 * g], a0, c0, c1);
                        mma16816_bf16(o[nt][2 * g + 1], a1, b0, b1);
                        mma16816_bf16(o[nt][2 * g + 1], a1, c0, c1);
                    }
                }
            }
            if (odd) {   // groups of V that stand for NaN, for the rows that see them
                for (int k = 0; k < kChunk; ++k) {
                    if (key0 + k >= a.hi || (gone >> (k >> 4) & 1)) continue;
                    const uint16_t *w = reinterpret_cast<const uint16_t *>(v_at + (k >> 4) * kBlock + kWordsAt + (k & 15) * quant_words(G));
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        if (!quant_is_nan<BITS>(w[g])) continue;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (key0 + k < sees[nt][i & 1]) o[nt][2 * g][i] = o[nt][2 * g + 1][i] = NAN;
                    }
                }
            }
            __syncwarp();   // the slot and the scratch are read
            if (next < t1) ask(slot);
            if (++slot == kSlots) {
                slot = 0;
                ++round;
            }
        }
        for (; !ok && pending > 0; --pending) {   // every copy must land
            mbar_drain(&s.full[warp][slot], round & 1);
            if (++slot == kSlots) {
                slot = 0;
                ++round;
            }
        }

        // ---------------------------------------------------- the warps' results
        const bool whole = t0 == 0 && t1 == a.steps;
        const int64_t out_slot = (int64_t)blockIdx.x * p.slots + (t0 == 0 ? kSlotLast : kSlotFirst);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            __syncthreads();   // every warp's ring is at rest, the rows before are read
            if (8 * nt >= a.rows) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (r8 == 0) s.stat[warp][2 * c + e] = make_float2(m[nt][e] * up, sum * 0x1p-24f);
                float *dst = s_out + (warp * 8 + 2 * c + e) * kOutRow;
#pragma unroll
                for (int g = 0; g < G; ++g) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ch = BITS == 4 ? 8 * (r8 >> 1) + 2 * i + (r8 & 1) : 4 * r8 + i;
                        dst[32 * g + ch] = o[nt][2 * g + (i >> 1)][2 * (i & 1) + e] * 0x1p-4f;
                    }
                }
            }
            __syncthreads();
            const int row = tid >> 4, r = 8 * nt + row;
            if (r >= a.rows) continue;
            float2 st[kWarps];
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                st[w] = s.stat[w][row];
                top = fmaxf(top, st[w].x);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            float weight[kWarps], sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                weight[w] = ex2(st[w].x - ref);
                sum = fmaf(st[w].y, weight[w], sum);
            }
            const bool see = attend_sees(p, a, r) > 0;
            const int64_t out_row = attend_out_row(p, a, r);
            const float inv = 1.f / sum;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int col = 32 * j + 2 * (tid & 15);
                float y0 = 0.f, y1 = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float *src = s_out + (w * 8 + row) * kOutRow + col;
                    y0 = fmaf(src[0], weight[w], y0);
                    y1 = fmaf(src[1], weight[w], y1);
                }
                if (whole) {
                    uint32_t both;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(both) : "f"(see ? y1 * inv : 0.f), "f"(see ? y0 * inv : 0.f));
                    *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + out_row * D + col) = both;
                } else {
                    *reinterpret_cast<float2 *>(p.part + (out_slot * p.slot_rows + r) * D + col) = make_float2(y0, y1);
                }
            }
            if ((tid & 15) == 0) {
                if (whole)
                    attend_store_lse(p, out_row, top, sum, see);
                else
                    p.stat[out_slot * p.slot_rows + r] = make_float2(top, sum);
            }
        }
        if (!whole) {
            const int c0 = attend_cta_of(run.total, run.grid, u_lo + p.extra);
            const int c1 = attend_cta_of(run.total, run.grid, u_lo + a.cost - 1);
            const int me = blockIdx.x, n = c1 - c0 + 1, groups = attend_groups(n);
            bool last = true;
            if (groups > 1) {
                const int g0 = c0 + (me - c0) / kJoinGroup * kJoinGroup, gn = min(kJoinGroup, c1 - g0 + 1);
                last = attend_block_last(&p.arrived[16 * g0 + 8], gn, &s.last);
                if (last)
                    attend_join<__nv_bfloat16, 2, 4>(p, a, AttendSpan{c0, g0, 1, gn, false, false}, 0, a.rows, 0, tid, kThreads);
            }
            if (last && attend_block_last(&p.arrived[16 * c0], groups > 1 ? groups : n, &s.last))
                attend_join<__nv_bfloat16, 2, 4>(p, a, AttendSpan{c0, c0, groups > 1 ? kJoinGroup : 1, groups > 1 ? groups : n, groups > 1, true},
                                                 0, a.rows, 0, tid, kThreads);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // bulk copies come after what was written here
        __syncthreads();   // the results are read: the ring may be filled again
        pos = end;
        u_lo += a.cost;
        u = attend_next(p, a, u);
    }
}

template <int G, int BITS, int NT>
int launch(AttendParams &p, int sms, cudaStream_t st) {
    constexpr size_t bytes = ring_bytes(BITS, G) + kWarps * scratch_bytes(G) + sizeof(Shared<slots_of(BITS, G)>);
    static_assert(bytes <= 232448, "shared memory of one block");
    allow_shared<attend_quant_kernel<G, BITS, NT>>((int)bytes);
    // as many blocks as an SM holds at once (1 KB of shared memory is each block's own cost)
    const int per_sm = std::max(1, std::min(per_sm_of(G, NT), (int)(233472 / (bytes + 1024))));
    launch_early(attend_quant_kernel<G, BITS, NT>, per_sm * sms, kThreads, bytes, st, p);
    return cache_launched(attend_name(p));
}

template <int G, int BITS>
int launch_rows(AttendParams &p, int rows, int sms, cudaStream_t st) {
    if (rows <= 8) return launch<G, BITS, 1>(p, sms, st);
    if constexpr (G == 2)
        if (rows > 16) return launch<G, BITS, 4>(p, sms, st);
    return launch<G, BITS, 2>(p, sms, st);
}

}  // namespace

int attend_quant_rows() { return 32; }

int launch_attend_quant(AttendParams &p, int rows, int sms, cudaStream_t st) {
    const char *skip = getenv("KVC_TEST_SKIP_ARRIVE");
    AttendParams own = p;
    own.skip_load = skip && skip[0] == '1';
    own.split_rows = 0;
    own.step_keys = kStepKeys;
    own.extra = kExtra;
    own.slots = 2;
    own.slot_rows = kSlotRows;
    // (two units of 16 rows for up to 32 of a head of 128, whose sums take the registers)
    const int unit = rows <= 8 ? 8 : rows <= 16 || p.dim == 128 ? 16 : 32;
    if (!attend_units(own, unit, 0, rows <= unit ? unit : 2 * unit)) {
        set_error("%s: n_seqs * n_kv_heads * max_new is too large", attend_name(p));
        return KVC_ERR_UNSUPPORTED;
    }
    if (p.bits == 4) return p.dim == 64 ? launch_rows<2, 4>(own, unit, sms, st) : launch_rows<4, 4>(own, unit, sms, st);
    return p.dim == 64 ? launch_rows<2, 8>(own, unit, sms, st) : launch_rows<4, 8>(own, unit, sms, st);
}

}  // namespace kvc
