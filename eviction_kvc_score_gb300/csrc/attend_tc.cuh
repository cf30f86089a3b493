// attend_tc.cuh -- attention of new tokens over the paged cache on the sm_103a
// tensor cores: bf16, head size 64 or 128, up to 128 query heads per KV head.
//
// A CTA walks its run of steps (attend.cuh).  Per 128-key tile of a list and
// per tile t of up to 128 rows (tokens x the KV head's query heads):
//   MMA   S_t = Q_t K^T        128 x 128, D deep, both operands in shared memory
//   soft  p = 2^(S c - m), c = scale log2 e, as two bf16 terms written over S_t
//         in TMEM: the upper 16 bits of p, and the rest rounded to bf16 (2^-16 p
//         is lost); l += sum of the unrounded p
//   MMA   O_t += P_t V         128 x D, both terms of P straight from TMEM, V as
//                              TMA left it (channel-contiguous: the MN-major layout)
// One term (KVC_ATTEND_BF16_P, the caller's choice) rounds p to 8 bits: the
// outputs' error against 64 bits is then 1.3 to 1.4 times that of an fp32 softmax
// rounded once; with two it is the same.  The second term costs half as many
// products again, and four instructions per pair of probabilities, which in a
// decode step one scheduler of four issues for both halves (their rows lie in the
// same quarter of TMEM): 16.9 us against 14.6 for one sequence of 1,000 rows, 170
// against 153 for the batch below, 1.99 ms against 1.41 for the chunk.
// The reference m only follows the running maximum when that has grown by more
// than 8 (p then stays below 2^8, far from any limit of bf16 or fp32); O and l
// are rescaled then, which after the first tiles hardly ever happens.
//
// Two row tiles share every K and V tile of a step (256 rows per read of the
// cache); while the softmax of one runs, the tensor cores work on the other.
// A unit of at most one tile's rows -- decode -- gives both halves the same
// rows and every other key tile each, so the two chains still overlap, and
// joins the halves at the end: 256 keys per step.
//
// Pages go to shared memory by TMA, one box of page_rows x 64 elements each;
// a page outside the pool is a box outside the tensor and comes as zeros.
// Nothing a row does not see reaches it: its S is masked, and in tiles that
// some row sees only part of, V's elements that are not finite are taken out
// before the product (p = 0 would not cancel them) and given back at the end
// to the rows that see them.  Elsewhere an infinite value goes through the
// product: neither term of a p above 2^-110 is 0 or negative.
//
// Roles: warps 0-3 and 4-7 softmax of t = 0 and 1, a thread per row; warps 8
// and 11 load, every other tile each (one warp takes 1,200 clocks to issue the
// 16 boxes of a tile of 16-row pages); warps 9 and 10 issue the MMAs of t = 0
// and 1 (one thread spent 4,300 clocks on the waits and MMAs of a step whose
// MMAs take 2,048).  Warp 8 also walks the units and puts segments of them into
// a queue for the others.  TMEM: S_0 | S_1 | O_0 | O_1, 128 columns each.  Shared
// memory: two Q tiles and a ring of 5 (D = 128: 64 + 160 KB) or 12 tiles that K
// and V pass through in the order the MMAs use them.  Every wait is bounded and
// nothing waits on a barrier without a limit, so a wait that runs out ends the
// kernel with KVC_DEV_TIMEOUT (the workspace then has to be initialised again).
//
// What bounds it, measured on one GB300:
// - chunks: the MMAs of a step of two halves take 3,072 clocks (128 x 128 x 16 in
//   64 clocks; one term: 2,048), the chain S -> softmax -> P V the rest.  4,096
//   tokens x 32 heads behind 28,672 cached rows: 1.99 ms back to back, 1,550
//   TFLOP/s of products or 91% of the measured sustained rate; one term 1.41.
// - decode: reading the cache, and the softmax of one warp between K and V.  64
//   sequences x 8 KV heads of 500-6,000 rows in 16-row pages, 853 MB: 170 us, 5.0
//   TB/s or 74% of the measured copy rate; one term 153 us, 82%.
// - short calls: latency.  One sequence of 1,000 rows: 16.9 us; one term 14.6.
//
// Rows held in 4 or 8 bits (BITS; quant.cuh; attend_tc_quant.cu): warps 12-19 make
// the tiles.  Warp 11 brings blocks of 16 rows to shared memory, a bulk copy each;
// each of the eight warps takes a block of every tile and writes it out as bf16, which
// holds (n - z) s exactly, in the layout that TMA would have left.  The rest is as with
// rows in bf16, two terms of P included; groups of V that stand for NaN are taken out by
// the warps that write the tile.  (V as fp16 over a power of two and P as one fp16 number
// took 216 us for the chunks and 1.95 ms for the long one below, but every power had to
// fit a tile's largest value: one seen by some tokens only took the others' bits.)
//
// What bounds them: the chain S -> softmax -> P V, whose softmax shares its issue slots
// with the writing of the tiles.  A step of two halves takes 6,300 clocks, twice what its
// MMAs take; of some 13,400 instructions a step (44% of the issue slots) the tiles are a
// third.  4,096 tokens x 32 heads over 32,768 rows in 4 bits: 2.47 ms, 833 TFLOP/s (rows in
// bf16: 1.99 ms); six chunks of 1-700 tokens over up to 5,700 rows in 8 bits 239 us, 438
// TFLOP/s; one term of P, 1.82 ms and 210 us.  Warps 12-19 and not the
// softmax's own: a step's tiles would then stand between its softmaxes.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "asked.cuh"
#include "attend.cuh"
#include "quant.cuh"

namespace kvc {

namespace {

// Registers per thread: 168 at launch (64,512 of the SM's 65,536), moved from
// the loading and issuing warpgroup to the two that hold a row of 128 logits
// per thread.  256 x 208 + 128 x 88 = 384 x 168: the launch checks the 168,
// because an increase beyond what the block was launched with never returns.
// With two warpgroups more: 256 x 152 + 128 x 64 + 256 x 56 = 640 x 96 (of what the
// softmax and the tiles share, 128 and 80 let the second term spill: a long chunk took
// 2.48 ms; 144 and 64 2.40, so 2.37).
template <int BITS>
struct Shape {
    static constexpr int kThreads = BITS == 0 ? 384 : 640;
    static constexpr int kRegsLaunch = BITS == 0 ? 168 : 96, kRegsSoftmax = BITS == 0 ? 208 : 152;
    static constexpr int kRegsOther = BITS == 0 ? 88 : 64, kRegsTiles = BITS == 0 ? 0 : 56;
    static_assert(256 * kRegsSoftmax + 128 * kRegsOther + 256 * kRegsTiles <= kThreads * kRegsLaunch, "register split");
    static constexpr int kReaders = BITS == 0 ? 12 : 20;   // warps that read the queue
};
constexpr int kTile = 128;              // rows of Q, keys of K and V
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLoadWarp2 = 11, kTileWarp = 12;
constexpr int kBox = kTile * 128;       // bytes of 128 rows x 64 bf16
constexpr uint32_t kColS = 0, kColO = 256;
constexpr float kGrow = 8.f;            // log2 units m may lag behind
constexpr int kSlotsTc = 2;
// A unit costs about 4 steps beside its steps (one term, 12 lists of 60,000-130,000
// rows: 68 us without, 63 with 4, 62 with 8; 512 short lists: 148, 150 and 152 us).
constexpr int kExtra = 4;
// One over held rows of 128 about 8 (us with 4, 8 and 12: 16 chunks of up to 300 tokens
// in 8 bits 302, 289, 296, in 4 bits 256, 252, 253, six of up to 700 234, 237, 234; of 64,
// with 2, 4 and 8, 32 chunks of up to 200: 166, 166, 172).  Units of one tile's rows, whose
// halves take every other key tile, would do with less (64 rows a list: 32 x 8 lists in 8
// bits 194, 222, 235, 64 x 8 in 4 bits 312, 317, 319).
constexpr int kExtraHeld = 8;
constexpr int kDirect = 4;              // shares that are joined from registers
constexpr int kQueue = 4;               // segments on their way from the walk to the roles

// What a CTA does of one unit: key tiles [first, first + n) of the list; half t
// takes cnt[t] of them, every one (paired) or every other (split).
struct Segment {
    bool split, whole, begins;   // begins: the unit's first step is in it
    int first, n, cnt[2];
    int c0, c1;              // the CTAs that share the unit
};

struct Work {
    AttendUnit a;
    Segment g;
    bool none;   // the run has ended
};

// Ring stages: what shared memory holds beside Q.
constexpr int stages_of(int kh, int bits) { return bits != 0 ? (kh == 2 ? 4 : 10) : kh == 2 ? 5 : 12; }
// Slots for blocks of 16 rows as they are held: whole tiles of them, so that a slot
// is always the same warp's.  (A warp that waited for a phase behind another warp's
// of the same slot would take the one before both for it: parities repeat.)
constexpr int raw_slots(int kh, int bits) { return bits == 0 ? 0 : bits == 4 ? 24 : kh == 2 ? 8 : 16; }
static_assert(raw_slots(1, 4) % 8 == 0 && raw_slots(2, 8) % 8 == 0 && raw_slots(1, 8) % 8 == 0, "eight blocks a tile");
constexpr int raw_bytes(int kh, int bits) { return bits == 0 ? 0 : raw_slots(kh, bits) * quant_block(bits, 2 * kh); }

template <int STAGES, int BITS, int RAW>
struct Bars {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2][2], o_full[2];   // p_full: [half][keys 0-63, 64-127]
    uint64_t half_full, half_empty, wg[2], joined[2], drain[2], issued[2];
    uint32_t tmem;
    volatile int abort_flag;
    int dirty;            // some value taken out of V
    int last[2][2];
    uint64_t work_full[kQueue], work_empty[kQueue];
    Work work[kQueue];
    float2 other[kTile];  // half 1's (max, sum) of a split unit
    int64_t plan[Shape<BITS>::kThreads / 32 + 4];
    // held rows: blocks that have come and gone
    uint64_t raw_full[BITS == 0 ? 1 : RAW], raw_empty[BITS == 0 ? 1 : RAW];
    volatile int raw_there[BITS == 0 ? 1 : RAW];   // blocks that a page of the pool holds
};

template <int KH, int BITS>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)(2 + stages_of(KH, BITS)) * KH * kBox + raw_bytes(KH, BITS) + sizeof(Bars<stages_of(KH, BITS), BITS, raw_slots(KH, BITS)>);
}

__device__ __forceinline__ void tma_load_4d(const CUtensorMap *map, uint64_t *bar, void *dst, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// O += P V: A (bf16 pairs along K) in TMEM, B in shared memory.
__device__ __forceinline__ void tc_mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                   uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Operand in the 128-byte swizzled layout TMA writes.  K-major: lbo unused,
// sbo between 8-row groups.  MN-major: lbo between blocks of 64 elements of MN,
// sbo between groups of 8 rows of K.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lbo >> 4) << 16 |
           static_cast<uint64_t>(sbo >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One thread of a converged warp, known to the compiler as such: the MMAs it
// issues take half as many clocks as those of a thread picked by its index.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

// The bounded wait, its outcome the same for the whole warp (what follows is
// warp-wide).  (Polling before the suspending wait cost 5% on a long chunk, by
// power: the SM clock fell from 1.69 to 1.54 GHz.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *stop,
                                          uint32_t *status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, stop, status));
}

// Slot of the k-th of the CTAs that share the segment's unit.
__device__ __forceinline__ int64_t share_at(const Segment &g, int k) {
    return (int64_t)(g.c0 + k) * kSlotsTc + (k == 0 ? kSlotLast : kSlotFirst);
}

// Eight floats at a 32-byte boundary, a whole sector, past L1.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    asm volatile("ld.global.cg.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store8(float *p, const float *v) {
    asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "l"(p)
                 : "memory");
}

__device__ __forceinline__ Segment segment_of(const AttendParams &p, const AttendUnit &a, int s0, int s1) {
    Segment g;
    g.split = a.rows <= p.split_rows;
    g.whole = s0 == 0 && s1 == a.steps;
    g.begins = s0 == 0;
    const int tiles = (a.hi + kTile - 1) / kTile;
    if (g.split) {
        g.first = 2 * s0;
        g.n = max(0, min(2 * s1, tiles) - g.first);
        g.cnt[0] = (g.n + 1) / 2;
        g.cnt[1] = g.n / 2;
    } else {
        const int t0 = (attend_sees(p, a, p.split_rows - 1) + kTile - 1) / kTile;
        g.first = s0;
        g.cnt[0] = max(0, min(s1, t0) - s0);
        g.cnt[1] = max(0, min(s1, tiles) - s0);
        g.n = g.cnt[1];
    }
    return g;
}

// Order of the ring: paired K0 V0 K1 V1 ..; split K0 K1 V0 K2 V1 K3 .. V.
__device__ __forceinline__ void load_at(const Segment &g, int l, bool *is_v, int *tile) {
    if (!g.split) {
        *is_v = l & 1;
        *tile = l >> 1;
        return;
    }
    const int lead = min(2, g.n), m = l - lead;
    if (m < 0) {
        *is_v = false;
        *tile = l;
    } else if (m < 2 * (g.n - lead)) {
        *is_v = !(m & 1);
        *tile = (m >> 1) + ((m & 1) ? 2 : 0);
    } else {
        *is_v = true;
        *tile = m - (g.n - lead);
    }
}
// Place in it of K and V of the segment's tile i.
__device__ __forceinline__ int k_at(const Segment &g, int i) {
    const int lead = min(2, g.n);
    return !g.split ? 2 * i : i < lead ? i : lead + 2 * (i - 2) + 1;
}
__device__ __forceinline__ int v_at(const Segment &g, int i) {
    return g.split ? min(2, g.n) + i + min(i, max(g.n - 2, 0)) : 2 * i + 1;
}

// Walks the units of the CTA's run.
template <bool kSome>
struct Walk {
    AttendRun run;
    int64_t pos, u_lo;
    int u;
    AttendRaw raw;   // of unit u, asked for while the unit before is worked on
    __device__ explicit Walk(const AttendRun &r)
        : run(r), pos(r.lo), u_lo(r.unit_lo), u(r.unit), raw(r.raw) {}
    __device__ void next(const AttendParams &p, Work &w) {
        w.none = true;
        while (w.none && pos < run.hi) {
            w.a = attend_unit<kSome>(p, u, raw);
            if (w.a.steps > 0) {
                const int64_t end = min(run.hi, u_lo + w.a.cost);
                const int s0 = max(0, (int)(pos - u_lo) - p.extra), s1 = max(0, (int)(end - u_lo) - p.extra);
                if (s1 > s0) {
                    w.g = segment_of(p, w.a, s0, s1);
                    w.g.c0 = attend_cta_of(run.total, run.grid, u_lo + p.extra);
                    w.g.c1 = attend_cta_of(run.total, run.grid, u_lo + w.a.cost - 1);
                    w.none = false;
                }
                pos = end;
                u_lo += w.a.cost;
            }
            u = w.a.steps > 0 ? attend_next(p, w.a, u) : attend_next_seq<kSome>(p, w.a.b);
            raw = attend_raw(p, u);
        }
    }
};

// 16 bytes of shared memory.
__device__ __forceinline__ void write16(uint32_t at, const uint32_t (&x)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
// A block of 16 rows as it is held, in a warp's registers: lane 4 j + c has piece c of
// all groups of rows r8 and r8 + 8, r8 = 0, 4, 1, 5, 2, 6, 3, 7 for j = 0 .. 7: the
// eight lanes whose 16 bytes are stored at a time hit eight places of the swizzle.
template <int KH, int BITS>
struct HeldRows {
    static constexpr int G = 2 * KH, kCodes = quant_codes(BITS, G);
    uint32_t word[2][KH];
    uint32_t code[2][kCodes / 16];

    static __device__ __forceinline__ int row8() { return (threadIdx.x >> 3 & 3) | (threadIdx.x & 4); }

    // Rows at and after `rows` are zeros.
    __device__ __forceinline__ void load(const uint8_t *raw, int rows) {
        const int r8 = row8(), c = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r8 + 8 * i;
            const uint8_t *w = raw + kQuantRows * kCodes + r * quant_words(G);
            if (KH == 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(w);
                word[i][0] = r < rows ? x.x : 0;
                word[i][KH - 1] = r < rows ? x.y : 0;
            } else {
                word[i][0] = r < rows ? *reinterpret_cast<const uint32_t *>(w) : 0;
            }
            const uint8_t *at = raw + r * kCodes + c * (kCodes / 4);
            if (kCodes == 32) {
                const uint2 x = *reinterpret_cast<const uint2 *>(at);
                code[i][0] = x.x;
                code[i][1] = x.y;
            } else {
#pragma unroll
                for (int k = 0; k < kCodes / 64; ++k) {
                    const uint4 x = reinterpret_cast<const uint4 *>(at)[k];
                    code[i][4 * k] = x.x;
                    code[i][4 * k + 1] = x.y;
                    code[i][4 * k + 2] = x.z;
                    code[i][4 * k + 3] = x.w;
                }
            }
        }
    }
    // The codes of group g of the i-th row.
    template <bool V>
    __device__ __forceinline__ uint2 piece(int i, int g) const {
        if (BITS == 8) return V ? make_uint2(code[i][g], code[i][G + g]) : make_uint2(code[i][2 * g], code[i][2 * g + 1]);
        if (!V) return make_uint2(code[i][g], 0);
        // halves of the group from two places
        return make_uint2(__byte_perm(code[i][g / 2], code[i][KH + g / 2], g & 1 ? 0x7632 : 0x5410), 0);
    }
    // V: groups that stand for NaN become zeros from row `finite` on; *dirty is set if
    // one of them is before `held`.
    __device__ __forceinline__ void clean(int finite, int held, volatile int *dirty) {
        constexpr uint32_t kExponent = BITS == 4 ? 0x7f80u : 0xff00u;
        uint32_t most = 0;   // of the upper and of the lower words
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KH; ++k) most = __vmaxu2(most, word[i][k] & (kExponent << 16 | kExponent));
        if (max(most >> 16, most & 0xffffu) != kExponent) return;
        const int r8 = row8();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KH; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if ((word[i][k] >> 16 * h & kExponent) == kExponent && r8 + 8 * i >= finite) {
                        word[i][k] &= h ? 0xffffu : 0xffff0000u;
                        if (r8 + 8 * i < held) *dirty = 1;
                    }
    }
    // To rows row0 .. + 15 of a tile.
    template <bool V>
    __device__ __forceinline__ void write(uint32_t tile, int row0) const {
        const int r8 = row8(), c = threadIdx.x & 3;
        const uint32_t at = tile + (row0 + r8) * 128 + ((c ^ r8) << 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KH; ++k) {
                const uint32_t w = word[i][k];
                uint32_t y0[4], y1[4];
                quant_bf16<BITS>(piece<V>(i, 2 * k), __byte_perm(w, 0, 0x1010), y0);
                quant_bf16<BITS>(piece<V>(i, 2 * k + 1), __byte_perm(w, 0, 0x3232), y1);
                const uint32_t to = at + i * 8 * 128 + k * kBox;
                write16(to, y0);
                write16(to ^ 0x40, y1);
            }
    }
};

// Bytes that are a multiple of 16 from global to shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int KH, bool TWO, int BITS>
__global__ void __launch_bounds__(Shape<BITS>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ AttendParams p) {
    constexpr int D = 64 * KH;
    constexpr int kStageBytes = KH * kBox, kStages = stages_of(KH, BITS), kThreads = Shape<BITS>::kThreads;
    constexpr bool kSome = BITS != 0;   // short lists may be another launch's
    extern __shared__ uint8_t raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sq = base;                              // [2][KH][128 rows][128 B]
    uint8_t *ring = base + 2 * kStageBytes;          // [stage][KH][128 keys][128 B]
    uint8_t *held = ring + kStages * kStageBytes;    // blocks as they are held
    constexpr int kRaw = raw_slots(KH, BITS);
    using Shared = Bars<kStages, BITS, kRaw>;
    Shared &b = *reinterpret_cast<Shared *>(held + raw_bytes(KH, BITS));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = p.split_rows;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&b.full[i], BITS == 0 ? 1 : 8);
            mbar_init(&b.empty[i], 2);
        }
        mbar_init(&b.q_full, 1);
        mbar_init(&b.q_empty, 2);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&b.s_full[t], 1);
            mbar_init(&b.p_full[t][0], 4);
            mbar_init(&b.p_full[t][1], 4);
            mbar_init(&b.o_full[t], 1);
            mbar_init(&b.wg[t], 1);
            mbar_init(&b.joined[t], 4);
            mbar_init(&b.drain[t], 1);
            mbar_init(&b.issued[t], 1);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(&b.work_full[i], 1);
            mbar_init(&b.work_empty[i], Shape<BITS>::kReaders);
        }
        if constexpr (BITS != 0)
            for (int i = 0; i < kRaw; ++i) {
                mbar_init(&b.raw_full[i], 1);
                mbar_init(&b.raw_empty[i], 1);
            }
        mbar_init(&b.half_full, 4);
        mbar_init(&b.half_empty, 4);
        b.abort_flag = 0;
        b.dirty = 0;
        fence_barrier_init();
    }
    let_next_start();
    wait_for_inputs();
    const AttendRun run = attend_plan<kThreads, kSome>(p, b.plan);
    if (run.lo >= run.hi) return;   // more CTAs than steps
    if (warp == kMmaWarp) {
        tmem_alloc(&b.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    volatile int *stop = &b.abort_flag;
    // Segment k of the run for a warp that reads the queue.  One warp walks the
    // units: the others would each pay for its loads, some 3 us between units
    // when memory is busy.
    auto read_work = [&](uint32_t k, Work &w) {
        const uint32_t e = k % kQueue;
        if (!warp_wait(&b.work_full[e], (k / kQueue) & 1, stop, p.status)) return false;
        w = b.work[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.work_empty[e]);
        return !w.none;
    };

    if (BITS != 0 && warp >= kTileWarp) {
        // ------------------------------------------------ tiles from rows as they are held
        if constexpr (BITS != 0) {
            regs_dec<Shape<BITS>::kRegsTiles>();
            constexpr int kBlock = quant_block(BITS, 2 * KH);
            const int part = warp - kTileWarp;   // keys 16 part .. of every tile
            uint32_t base_fill = 0;         // loads before this segment
            uint32_t slot = part, round = 0;   // of the block that is next
            bool ok = true;
            Work w;
            for (uint32_t k = 0; ok; ++k) {
                if (!read_work(k, w)) break;
                const Segment g = w.g;
                const int hi = w.a.hi, from = attend_sees(p, w.a, 0), len = w.a.len;
                const int key0 = g.first * kTile + kQuantRows * part;
                HeldRows<KH, BITS> rows;
                bool is_v = false;
                int tile = 0;
                // load l's rows to registers; their slot is free again
                auto read = [&](int l) {
                    load_at(g, l, &is_v, &tile);
                    if (!warp_wait(&b.raw_full[slot], round & 1, stop, p.status)) return false;
                    rows.load(held + slot * kBlock, b.raw_there[slot] ? hi - (key0 + tile * kTile) : 0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.raw_empty[slot]);
                    if ((slot += 8) >= kRaw) {
                        slot -= kRaw;
                        ++round;
                    }
                    return true;
                };
                if (g.n > 0) ok = read(0);
                for (int l = 0; ok && l < 2 * g.n; ++l) {
                    const uint32_t fill = base_fill + l, st = fill % kStages;
                    if (!(ok = fill < kStages || warp_wait(&b.empty[st], (fill / kStages - 1) & 1, stop, p.status))) break;
                    const uint32_t to = smem_u32(ring) + st * kStageBytes;
                    if (is_v) {
                        const int key = key0 + tile * kTile;
                        rows.clean(from - key, len - key, &b.dirty);
                        rows.template write<true>(to, kQuantRows * part);
                    } else {
                        rows.template write<false>(to, kQuantRows * part);
                    }
                    if (l + 1 < 2 * g.n) ok = read(l + 1);
                    __threadfence_block();   // what was taken out is noted
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && !(p.skip_load && fill == 0)) mbar_arrive(&b.full[st]);
                }
                base_fill += 2 * g.n;
            }
        }
    } else if (warp >= kLoadWarp) {
    regs_dec<Shape<BITS>::kRegsOther>();
    if (BITS != 0 && warp == kLoadWarp) {
        // ------------------------------------------------ the walk, and Q
        if (lane == 0) tma_prefetch_desc(&tq);
        Walk<kSome> walk(run);
        uint32_t segs = 0;
        bool ok = true;
        Work w;
        for (uint32_t k = 0; ok; ++k) {
            const uint32_t e = k % kQueue;
            walk.next(p, w);
            if (k >= kQueue && !warp_wait(&b.work_empty[e], (k / kQueue - 1) & 1, stop, p.status)) break;
            if (lane == 0) {
                b.work[e] = w;
                mbar_arrive(&b.work_full[e]);
                mbar_arrive(&b.work_empty[e]);   // this warp has read it
            }
            if (w.none) break;
            if (w.g.n == 0) continue;
            ok = segs == 0 || warp_wait(&b.q_empty, (segs - 1) & 1, stop, p.status);
            if (!ok) break;
            if (lane == 0) {
                const int tiles = w.g.split ? 1 : 2;
                mbar_arrive_expect_tx(&b.q_full, (uint32_t)(tiles * KH * R * 128));
                for (int t = 0; t < tiles; ++t)
                    for (int kh = 0; kh < KH; ++kh)
                        tma_load_4d(&tq, &b.q_full, sq + t * kStageBytes + kh * kBox, kh * 64, 0, w.a.h,
                                    w.a.q0 + p.by_group(w.a.row0 + t * R));
            }
            ++segs;
        }
        if (*stop && segs) mbar_drain(&b.q_full, (segs - 1) & 1);
    } else if (BITS != 0 && warp == kLoadWarp2) {
        // ------------------------------------------------ rows as they are held, a block a lane
        if constexpr (BITS != 0) {
            constexpr int kBlock = quant_block(BITS, 2 * KH);
            uint32_t asked = lane & 7;   // lanes 0-7: the tile's eight blocks
            bool ok = true;
            Work w;
            for (uint32_t k = 0; ok; ++k) {
                if (!read_work(k, w)) break;
                const Segment &g = w.g;
                const int hi = w.a.hi;
                const int32_t *entry = p.table + (int64_t)w.a.list * p.max_pages;
                // page numbers of four tiles, a lane each; those of the next four are asked
                // for ahead, those before are kept: V is up to two tiles behind K
                auto look_up = [&](int batch) {
                    const int64_t key = (int64_t)(g.first + batch * 4) * kTile + 16 * lane;
                    return key < hi ? entry[key >> p.shift] : 0;
                };
                int batch = 0, before = 0, now = 0, then = 0;
                if (g.n > 0) {
                    now = look_up(0);
                    then = look_up(1);
                }
                for (int l = 0; l < 2 * g.n; ++l) {
                    bool is_v;
                    int tile;
                    load_at(g, l, &is_v, &tile);
                    if (tile >> 2 > batch) {
                        ++batch;
                        before = now;
                        now = then;
                        then = look_up(batch + 1);
                    }
                    const int page = __shfl_sync(0xffffffffu, tile >> 2 < batch ? before : now, (tile & 3) * 8 + (lane & 7));
                    const int key = (g.first + tile) * kTile + 16 * (lane & 7);
                    const bool seen = key < hi, there = seen && page >= 0 && page < p.n_pages;
                    const uint32_t slot = asked % kRaw;
                    const bool mine = lane < 8;
                    bool free = true;
                    if (mine && asked >= kRaw) free = mbar_wait(&b.raw_empty[slot], (asked / kRaw - 1) & 1, stop, p.status);
                    if (!(ok = __all_sync(0xffffffffu, free))) break;
                    if (mine) {
                        b.raw_there[slot] = there;
                        if (there) {
                            const int64_t block = (((int64_t)page << p.shift) + (key & ((1 << p.shift) - 1))) >> 4;
                            mbar_arrive_expect_tx(&b.raw_full[slot], kBlock);
                            bulk_load(held + slot * kBlock, static_cast<const uint8_t *>(is_v ? p.v_pool : p.k_pool) + block * kBlock, kBlock,
                                      &b.raw_full[slot]);
                        } else {
                            if (seen) set_status(p.status, KVC_DEV_BAD_PAGE);
                            mbar_arrive(&b.raw_full[slot]);
                        }
                    }
                    asked += 8;
                }
            }
            if (*stop && lane < 8) {   // unwind: every copy must land
                const uint32_t all = asked - lane, first = all > kRaw ? all - kRaw : 0;   // the last of each slot
                for (uint32_t i = lane; i < asked; i += 8)
                    if (i >= first) mbar_drain(&b.raw_full[i % kRaw], (i / kRaw) & 1);
            }
        }
    } else if (BITS == 0 && (warp == kLoadWarp || warp == kLoadWarp2)) {
        // ------------------------------------------------ loads, every other one a warp
        const uint32_t side = warp == kLoadWarp ? 0 : 1;
        if (lane == 0) {
            tma_prefetch_desc(&tq);
            tma_prefetch_desc(&tk);
            tma_prefetch_desc(&tv);
        }
        uint32_t base_fill = 0, segs = 0, done = 0;   // loads before this segment, segments, loads of this side
        bool ok = true;
        const int tile_shift = 7 - p.shift, per_tile = 1 << tile_shift, ps = 1 << p.shift;
        Walk<kSome> walk(run);
        uint32_t put = 0;   // segments in the queue so far
        auto put_work = [&]() {
            const uint32_t e = put % kQueue;
            Work w;
            walk.next(p, w);
            if (put >= kQueue && !warp_wait(&b.work_empty[e], (put / kQueue - 1) & 1, stop, p.status)) return false;
            if (lane == 0) {
                b.work[e] = w;
                mbar_arrive(&b.work_full[e]);
            }
            ++put;
            return true;
        };
        if (side == 0) ok = put_work();
        Work w;
        for (uint32_t k = 0; ok; ++k) {
            if (!read_work(k, w)) break;
            const Segment &g = w.g;
            bool ahead = side != 0;   // the next segment is in the queue
            if (g.n == 0) {
                if (!ahead) ok = put_work();
                continue;
            }
            if (side == 0) {   // Q once the segment before has used it
                ok = segs == 0 || warp_wait(&b.q_empty, (segs - 1) & 1, stop, p.status);
                if (!ok) break;
                if (lane == 0) {
                    const int tiles = g.split ? 1 : 2;
                    mbar_arrive_expect_tx(&b.q_full, (uint32_t)(tiles * KH * R * 128));
                    for (int t = 0; t < tiles; ++t)
                        for (int kh = 0; kh < KH; ++kh)
                            tma_load_4d(&tq, &b.q_full, sq + t * kStageBytes + kh * kBox, kh * 64, 0, w.a.h,
                                        w.a.q0 + p.by_group(w.a.row0 + t * R));
                }
                ++segs;
            }
            // page numbers 32 at a time, a lane each: the batch in use, the
            // one before (V is up to two tiles behind K) and the next, asked
            // for while the one in use lasts
            const int page0 = g.first << tile_shift;
            const int page1 = min((g.first + g.n) << tile_shift, (w.a.hi + ps - 1) >> p.shift);
            auto look_up = [&](int batch) {
                const int j = page0 + batch * 32 + lane;
                return j < page1 ? p.table[(int64_t)w.a.list * p.max_pages + j] : 0;
            };
            int batch = 0, before = 0, now = look_up(0), then = look_up(1);
            // a segment makes an even number of loads: the sides keep their parity
            for (int l = (int)side; l < 2 * g.n; l += 2) {
                bool is_v;
                int tile;
                load_at(g, l, &is_v, &tile);
                const int at = tile << tile_shift;   // the tile's first page, within the segment
                if (at >> 5 > batch) {
                    ++batch;
                    before = now;
                    now = then;
                    then = look_up(batch + 1);
                }
                int page = __shfl_sync(0xffffffffu, at >> 5 < batch ? before : now, (at + lane) & 31);
                // those that hold visible rows
                const int pages = min(per_tile, page1 - page0 - at);
                if (lane < pages && (page < 0 || page >= p.n_pages)) {
                    set_status(p.status, KVC_DEV_BAD_PAGE);
                    page = p.n_pages;   // outside the tensor: zeros
                }
                const uint32_t fill = base_fill + l, st = fill % kStages;
                ok = fill < kStages || warp_wait(&b.empty[st], (fill / kStages - 1) & 1, stop, p.status);
                if (!ok) break;
                if (p.skip_load && fill == 0) {   // nobody fills this stage
                    ++done;
                    continue;
                }
                if (lane == 0) mbar_arrive_expect_tx(&b.full[st], (uint32_t)(pages * ps * D * 2));
                __syncwarp();
                if (lane < pages) {
                    uint8_t *dst = ring + st * kStageBytes + (lane << p.shift) * 128;
#pragma unroll
                    for (int kh = 0; kh < KH; ++kh)
                        tma_load_3d(is_v ? &tv : &tk, &b.full[st], dst + kh * kBox, kh * 64, 0, page);
                }
                ++done;
                // the ring is full or the segment done: time for the next one
                if (!ahead && (l + 2 >= kStages || l + 2 >= 2 * g.n)) {
                    ahead = true;
                    if (!(ok = put_work())) break;
                }
            }
            base_fill += 2 * g.n;
        }
        if (*stop) {   // unwind: every copy started must land
            for (uint32_t i = done > (kStages + 1) / 2 ? done - (kStages + 1) / 2 : 0; i < done; ++i) {
                const uint32_t f = 2 * i + side;
                mbar_drain(&b.full[f % kStages], (f / kStages) & 1);
            }
            if (segs) mbar_drain(&b.q_full, (segs - 1) & 1);
        }
    } else if (warp >= kMmaWarp && warp < kMmaWarp + 2) {
        // ------------------------------------------------ MMA issue, a warp per half
        if (elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16_f32(kTile, kTile);
            constexpr uint32_t kIdO = idesc_bf16_f32(kTile, D) | (1u << 16);   // B MN-major
            const int t = warp - kMmaWarp;
            const uint32_t col_s = tmem + kColS + t * 128, col_o = tmem + kColO + t * 128;
            uint32_t use = 0, segs = 0, np = 0;   // ring stages passed, segments, P tiles seen
            uint32_t turns = 0;                   // groups of MMAs that both halves issue in turn
            auto stage_full = [&](uint32_t f) {
                return mbar_wait(&b.full[f % kStages], (f / kStages) & 1, stop, p.status);
            };
            // a stage is free after two arrivals: this half's commit, and the
            // other's or, of a tile that only this half uses, a plain one
            auto stage_used = [&](uint32_t f, bool alone) {
                if (alone) mbar_arrive(&b.empty[f % kStages]);
                tc_commit(&b.empty[f % kStages]);
            };
            auto issue_s = [&](bool split, uint32_t f) {
                const uint64_t a = desc_sw128(smem_u32(sq) + (split ? 0 : t * kStageBytes), 16, 1024);
                const uint64_t k = desc_sw128(smem_u32(ring) + (f % kStages) * kStageBytes, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < 4 * KH; ++ks) {
                    const uint64_t off = (uint64_t)(((ks >> 2) * kBox + (ks & 3) * 32) >> 4);
                    tc_mma_bf16(col_s, a + off, k + off, kIdS, ks > 0);
                }
                tc_commit(&b.s_full[t]);
            };
            // keys 0-63 or 64-127 of the tile; the first group of a unit's first tile does not
            // add.  (Held rows: the upper ones come first, and each 64 keys' P lies over their
            // own S, the second term behind the first.)
            auto issue_o = [&](uint32_t f, auto second, bool add) {
                constexpr bool kUpper = decltype(second)::value == (BITS == 0);
                constexpr int k0 = kUpper ? 4 : 0, kP = BITS != 0 && kUpper ? 32 : 0, kSecond = BITS != 0 ? 32 : 64;
                const uint64_t v = desc_sw128(smem_u32(ring) + (f % kStages) * kStageBytes, kBox, 1024);
#pragma unroll
                for (int ks = k0; ks < k0 + 4; ++ks) {
                    const uint64_t at = v + (uint64_t)(ks * (16 * 128 >> 4));
                    tc_mma_bf16_tmem_a(col_o, col_s + kP + ks * 8, at, kIdO, add || ks > k0);
                    if (TWO) tc_mma_bf16_tmem_a(col_o, col_s + kP + kSecond + ks * 8, at, kIdO, 1);
                }
            };
            // The halves' groups (O of a tile, S of the next) go to the tensor
            // cores whole and in turn.  Mixed, both softmaxes would get their S
            // at the same time and the tensor cores would wait for both
            // (measured: a step of 4,930 clocks).
            auto my_turn = [&]() {
                return t == 0 ? turns == 0 || mbar_wait(&b.issued[1], (turns - 1) & 1, stop, p.status)
                              : mbar_wait(&b.issued[0], turns & 1, stop, p.status);
            };
            auto turn_over = [&]() {
                mbar_arrive(&b.issued[t]);
                ++turns;
            };
            bool ok = true;
            Work w;
            for (uint32_t k = 0; ok; ++k) {
                if (!(ok = mbar_wait(&b.work_full[k % kQueue], (k / kQueue) & 1, stop, p.status))) break;
                w = b.work[k % kQueue];
                mbar_arrive(&b.work_empty[k % kQueue]);
                if (w.none) break;
                const Segment &g = w.g;
                if (g.n == 0) continue;
                if (!(ok = mbar_wait(&b.q_full, segs & 1, stop, p.status))) break;
                ++segs;
                tc_fence_after();
                const int cnt = g.cnt[t], both = min(g.cnt[0], g.cnt[1]);
                if (cnt == 0) mbar_arrive(&b.q_empty);
                for (int i = 0; i < cnt; ++i) {
                    const int ti = g.split ? 2 * i + t : i;
                    const bool alone = g.split || i >= g.cnt[t ^ 1];
                    if (i == 0) {
                        const uint32_t f = use + k_at(g, ti);
                        if (!(ok = stage_full(f))) break;
                        if (both > 0 && !(ok = my_turn())) break;
                        tc_fence_after();
                        issue_s(g.split, f);
                        if (both > 0) turn_over();
                        stage_used(f, alone);
                        if (cnt == 1) tc_commit(&b.q_empty);
                    }
                    const uint32_t fv = use + v_at(g, ti);
                    const bool more = i + 1 < cnt;
                    if (!(ok = stage_full(fv))) break;
                    const uint32_t fk = more ? use + k_at(g, g.split ? ti + 2 : ti + 1) : 0;
                    if (more && !(ok = stage_full(fk))) break;
                    if (!(ok = mbar_wait(&b.p_full[t][0], np & 1, stop, p.status))) break;
                    if (i < both && !(ok = my_turn())) break;
                    tc_fence_after();
                    issue_o(fv, std::false_type{}, i > 0);
                    if (!(ok = mbar_wait(&b.p_full[t][1], np & 1, stop, p.status))) break;
                    ++np;
                    tc_fence_after();
                    issue_o(fv, std::true_type{}, true);
                    if (more) issue_s(g.split, fk);
                    if (i < both) turn_over();
                    if (more) {
                        stage_used(fv, alone);
                        stage_used(fk, g.split || i + 1 >= g.cnt[t ^ 1]);
                        if (i + 2 == cnt) tc_commit(&b.q_empty);
                    } else {
                        tc_commit(&b.o_full[t]);
                        stage_used(fv, alone);
                    }
                }
                use += 2 * g.n;
            }
            tc_commit(&b.drain[t]);
            mbar_drain(&b.drain[t], 0);
        }
    }
    } else {
        // ------------------------------------------------ softmax and output
        regs_inc<Shape<BITS>::kRegsSoftmax>();
        const int t = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;   // row of the tile
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t cs = tmem + lanes + kColS + t * 128, co = tmem + lanes + kColO + t * 128;
        // whole tiles take maxima of S itself: only for a positive factor
        const bool plain = p.scale_log2 > 0.f;
        const float c = p.scale_log2;
        const unsigned long long c2 = f2_pack(c, c);
        // p (1 + 2^-23): the second term of a p > 0 is never 0, which an infinite value of V may not meet
        const unsigned long long above1 = f2_pack(1.f + 0x1p-23f, 1.f + 0x1p-23f);
        uint32_t ns = 0, no = 0, nwg = 0, njoined = 0, handed = 0, filled = 0;
        bool owed = false;   // half 1: O is still being read by half 0
        bool ok = true;
        Work w;
        for (uint32_t k = 0; ok; ++k) {
            if (!read_work(k, w)) break;
            const AttendUnit &a = w.a;
            const Segment &g = w.g;
            const int rt = g.split ? r : t * R + r;
            const bool real = r < R && rt < a.rows;
            const bool any = __any_sync(0xffffffffu, real);
            const int sees = real ? attend_sees(p, a, rt) : 0;
            int sees0 = attend_sees(p, a, g.split ? 0 : t * R);   // the tile's first row's
            const int from = attend_sees(p, a, 0);                      // the unit's
            float m = -INFINITY, l = 0.f;
            const int cnt = g.cnt[t];
            for (int i = 0; i < cnt; ++i) {
                const int ti = g.split ? 2 * i + t : i;
                const int k0 = (g.first + ti) * kTile;
                if (!(ok = warp_wait(&b.s_full[t], ns & 1, stop, p.status))) break;
                ++ns;
                tc_fence_after();
                const bool edge = k0 + kTile > sees0;
                if (owed) {
                    if (!(ok = warp_wait(&b.half_empty, (handed - 1) & 1, stop, p.status))) break;
                    owed = false;
                }
                if (BITS == 0 && k0 + kTile > from) {
                    // V's rows from the first that some row of the unit does
                    // not see.  Both halves go over the same rows, so each
                    // product finds them clean whatever the other half is at;
                    // the note that something was taken out comes first.
                    const uint32_t f = filled + v_at(g, ti);
                    if (!(ok = warp_wait(&b.full[f % kStages], (f / kStages) & 1, stop, p.status))) break;
                    if (k0 + r >= from) {
                        uint8_t *row = ring + (f % kStages) * kStageBytes + r * 128;
                        // a halfword of ~x & 0x7f80 is 0 where x is not finite;
                        // lanes start at chunks of their own: no bank conflicts
                        uint32_t low = 0xffffffffu;
#pragma unroll
                        for (int ch = 0; ch < 8 * KH; ++ch) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(row + (ch >> 3) * kBox + ((ch + r) & 7) * 16);
                            low = __vminu2(__vminu2(__vminu2(low, ~x.x & 0x7f807f80u), ~x.y & 0x7f807f80u),
                                           __vminu2(~x.z & 0x7f807f80u, ~x.w & 0x7f807f80u));
                        }
                        if ((low & 0xffffu) == 0 || (low >> 16) == 0) {
                            if (k0 + r < a.len) *static_cast<volatile int *>(&b.dirty) = 1;
                            __threadfence_block();
                            for (int e = 0; e < 32 * KH; ++e) {
                                uint32_t *at = reinterpret_cast<uint32_t *>(row + (e >> 5) * kBox + (e & 31) * 4);
                                uint32_t x = *at;
                                if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                                if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                                *at = x;
                            }
                        }
                    }
                    fence_async_shared();
                    // lane 0 says for all 32 rows that they are clean
                    __syncwarp();
                }
                // slow: some row of the tile sees only part of it, or the scale is
                // not positive; two copies, because a select per logit costs as much
                // as the rest.  The other way takes S c - m in one step, which is 2^-24 of m
                // off the product m: a row whose m would be beyond 2^24 goes the slow way, where
                // S c is rounded as m was, and the other returns without having done anything.
                auto far = [&](float top) { return __any_sync(0xffffffffu, sees > 0 && fabsf(top) > 0x1p24f); };
                auto soften = [&](auto slow) {
                    constexpr bool kSlow = decltype(slow)::value;
                    unsigned long long mul2 = c2;
                    float mul = c;
                    float v[4][32];
                    const int lim = sees - k0;   // keys of the tile the row sees
                    float x[4];
                    tmem_ld32(cs, v[0]);
                    tmem_ld32(cs + 32, v[1]);
                    tmem_ld_wait();
                    reg_fence(v[0]);
                    reg_fence(v[1]);
                    // the second half is on its way during the first one's maximum
                    tmem_ld32(cs + 64, v[2]);
                    tmem_ld32(cs + 96, v[3]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q == 2) {
                            tmem_ld_wait();
                            reg_fence(v[2]);
                            reg_fence(v[3]);
                        }
                        if (kSlow) {
                            // scaled here: -infinity for what is not seen may not
                            // meet a factor of 0 or below later
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[q][j] = q * 32 + j < lim ? v[q][j] * p.scale_log2 : -INFINITY;
                        }
                        x[q] = fmax3(v[q][0], v[q][1], v[q][2]);
#pragma unroll
                        for (int j = 3; j < 31; j += 2) x[q] = fmax3(x[q], v[q][j], v[q][j + 1]);
                        x[q] = fmaxf(x[q], v[q][31]);
                    }
                    if (kSlow) {
                        mul = 1.f;
                        mul2 = f2_pack(1.f, 1.f);
                    }
                    const float s_top = fmaxf(fmax3(x[0], x[1], x[2]), x[3]);
                    const float top = s_top * mul;
                    const bool grow = top > m + kGrow;
                    if (i == 0 || __any_sync(0xffffffffu, grow)) {
                        if (!kSlow && far(top)) return false;
                        if (i == 0) {
                            m = top;
                        } else {
                            // every product of this half up to the tile before is done: S came after it
                            const float down = grow ? ex2(m - top) : 1.f;
                            if (grow) m = top;
                            l *= down;
#pragma unroll 1
                            for (int d = 0; d < D; d += 32) {
                                float o[32];
                                uint32_t ou[32];
                                tmem_ld32(co + d, o);
                                tmem_ld_wait();
                                reg_fence(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) ou[j] = __float_as_uint(o[j] * down);
                                tmem_st32(co + d, ou);
                            }
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
                    const unsigned long long nm2 = f2_pack(nm, nm);
                    unsigned long long sum2[2] = {0, 0};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pw[32];
                        [[maybe_unused]] uint32_t lo[TWO ? 32 : 1];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int q = 2 * h + (j >> 4), e = 2 * (j & 15);
                            float y0, y1;
                            f2_unpack(f2_fma(f2_pack(v[q][e], v[q][e + 1]), mul2, nm2), y0, y1);
                            const float p0 = ex2(y0), p1 = ex2(y1);
                            const unsigned long long pp = f2_pack(p0, p1);
                            sum2[j & 1] = f2_add(sum2[j & 1], pp);
                            if constexpr (TWO) {
                                // the upper 16 bits, and what is left of the rest
                                const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                                pw[j] = __byte_perm(b0, b1, 0x7632);
                                float r0, r1;
                                f2_unpack(f2_fma(pp, above1, f2_pack(-__uint_as_float(b0 & 0xffff0000u),
                                                                     -__uint_as_float(b1 & 0xffff0000u))),
                                          r0, r1);
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo[j]) : "f"(r1), "f"(r0));
                            } else {
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pw[j]) : "f"(p1), "f"(p0));
                            }
                        }
                        tmem_st32(cs + h * 32, pw);
                        if constexpr (TWO) tmem_st32(cs + 64 + h * 32, lo);   // S is in registers by now
                        // half of P is enough for half of the product to start
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b.p_full[t][h]);
                        if (h == 0) {   // not earlier: the first half's exponentials come first
                            reg_fence(v[2]);
                            reg_fence(v[3]);
                        }
                    }
                    float s0, s1;
                    f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
                    l += s0 + s1;
                    return true;
                };
                // held rows: 64 logits at a time for want of registers.  The maximum of
                // keys 0-63, that of keys 64-127, whose probabilities come first, and then
                // keys 0-63 once more.
                auto soften_held = [&](auto slow) {
                    constexpr bool kSlow = decltype(slow)::value;
                    const int lim = sees - k0;
                    auto seen = [&](int j, float s) { return j < lim ? s * c : -INFINITY; };
                    float v[2][32], x[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tmem_ld32(cs + 64 * h, v[0]);
                        tmem_ld32(cs + 64 * h + 32, v[1]);
                        tmem_ld_wait();
                        reg_fence(v[0]);
                        reg_fence(v[1]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float(&y)[32] = v[q];
                            if (kSlow) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) y[j] = seen(64 * h + 32 * q + j, y[j]);
                            }
                            float &top = x[2 * h + q];
                            top = fmax3(y[0], y[1], y[2]);
#pragma unroll
                            for (int j = 3; j < 31; j += 2) top = fmax3(top, y[j], y[j + 1]);
                            top = fmaxf(top, y[31]);
                        }
                    }
                    const float top = fmaxf(fmax3(x[0], x[1], x[2]), x[3]) * (kSlow ? 1.f : c);
                    const bool grow = top > m + kGrow;
                    if (i == 0 || __any_sync(0xffffffffu, grow)) {
                        if (!kSlow && far(top)) return false;
                        if (i == 0) {
                            m = top;
                        } else {
                            const float down = grow ? ex2(m - top) : 1.f;
                            if (grow) m = top;
                            l *= down;
#pragma unroll 1
                            for (int d = 0; d < D; d += 16) {
                                float o[16];
                                uint32_t ou[16];
                                tmem_ld16(co + d, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    asm volatile("" : "+f"(o[j]));   // read once it is there
                                    ou[j] = __float_as_uint(o[j] * down);
                                }
                                tmem_st16(co + d, ou);
                            }
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
                    const unsigned long long nm2 = f2_pack(nm, nm);
                    unsigned long long sum2[2] = {0, 0};
                    // keys 32 q .. + 31 of the tile from y, the slow way already scaled or not
                    auto weigh = [&](int q, float(&y)[32], auto scaled) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t pw[8];
                            [[maybe_unused]] uint32_t lo[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                float y0 = y[16 * h + 2 * j], y1 = y[16 * h + 2 * j + 1];
                                if (kSlow) {
                                    if (!decltype(scaled)::value) {
                                        y0 = seen(q * 32 + 16 * h + 2 * j, y0);
                                        y1 = seen(q * 32 + 16 * h + 2 * j + 1, y1);
                                    }
                                    f2_unpack(f2_add(f2_pack(y0, y1), nm2), y0, y1);
                                } else {
                                    f2_unpack(f2_fma(f2_pack(y0, y1), c2, nm2), y0, y1);
                                }
                                const float p0 = ex2(y0), p1 = ex2(y1);
                                const unsigned long long pp = f2_pack(p0, p1);
                                sum2[j & 1] = f2_add(sum2[j & 1], pp);
                                if constexpr (TWO) {
                                    // the upper 16 bits, and what is left of the rest
                                    const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                                    pw[j] = __byte_perm(b0, b1, 0x7632);
                                    float r0, r1;
                                    f2_unpack(f2_add(pp, f2_pack(-__uint_as_float(b0 & 0xffff0000u), -__uint_as_float(b1 & 0xffff0000u))), r0, r1);
                                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo[j]) : "f"(r1), "f"(r0));
                                } else {
                                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pw[j]) : "f"(p1), "f"(p0));
                                }
                            }
                            // over logits that are in registers or read for the last time
                            const uint32_t to = cs + (q < 2 ? 0 : 32) + 16 * q + 8 * h;
                            tmem_st8(to, pw);
                            if constexpr (TWO) tmem_st8(to + 32, lo);
                        }
                    };
                    auto handed = [&](int h) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b.p_full[t][h]);
                    };
                    weigh(2, v[0], std::true_type{});
                    tmem_ld32(cs, v[0]);
                    weigh(3, v[1], std::true_type{});
                    tmem_ld32(cs + 32, v[1]);
                    handed(0);
                    tmem_ld_wait();
                    reg_fence(v[0]);
                    reg_fence(v[1]);
                    weigh(0, v[0], std::false_type{});
                    weigh(1, v[1], std::false_type{});
                    handed(1);
                    float s0, s1;
                    f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
                    l += s0 + s1;
                    return true;
                };
                if (any) {
                    bool slow = edge || !plain;
                    if constexpr (BITS != 0) {
                        if (!slow && !soften_held(std::false_type{})) {
                            slow = true;
                            sees0 = 0;   // and the tiles behind it
                        }
                        if (slow) soften_held(std::true_type{});
                    } else {
                        if (!slow && !soften(std::false_type{})) {
                            slow = true;
                            sees0 = 0;
                        }
                        if (slow) soften(std::true_type{});
                    }
                } else if (lane == 0) {
                    mbar_arrive(&b.p_full[t][0]);
                    mbar_arrive(&b.p_full[t][1]);
                }
            }
            if (!ok) break;
            if (cnt > 0) {
                if (!(ok = warp_wait(&b.o_full[t], no++ & 1, stop, p.status))) break;
                tc_fence_after();
            }
            filled += 2 * g.n;
            if (g.split && t == 1) {
                // the other half takes these rows over, O straight from TMEM
                if (cnt > 0) {
                    b.other[r] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.half_full);
                    ++handed;
                    owed = true;
                }
                continue;
            }
            const bool take = g.split && g.cnt[1] > 0;
            float w_mine = 1.f, w_other = 0.f;
            if (take) {
                if (!(ok = warp_wait(&b.half_full, handed++ & 1, stop, p.status))) break;
                tc_fence_after();
                const float2 st = b.other[r];
                const float top = fmaxf(m, st.x), ref = top == -INFINITY ? 0.f : top;
                w_mine = ex2(m - ref);
                w_other = ex2(st.x - ref);
                l = l * w_mine + st.y * w_other;
                m = top;
            }
            const int64_t slot = ((int64_t)blockIdx.x * kSlotsTc + (g.begins ? kSlotLast : kSlotFirst)) * p.slot_rows +
                                 t * kTile + r;
            const int n = g.whole ? 1 : g.c1 - g.c0 + 1, me = (int)blockIdx.x;
            const int rows = min(a.rows - t * R, R);   // of the tile
            uint32_t *of_unit = &p.arrived[16 * g.c0 + 4 * t + (rows > 32 ? quarter : 0)];
            // The others of a few are all done (mostly: the CTA that begins a
            // unit ends with it, long after the others did their share): join
            // from the registers, without writing this share down.  The sums
            // are attend_join's, term by term.  (Tiles of few rows, where the
            // look costs more than the writing, do without.)
            bool direct = false;
            float weight[kDirect];
            if (!g.whole && n <= kDirect && rows > 32 && any) {
                direct = attend_peek(of_unit) == (uint32_t)(n - 1);
                if (direct) {
                    float2 st[kDirect];
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kDirect; ++k) {
                        st[k] = make_float2(-INFINITY, 0.f);
                        if (k < n) st[k] = g.c0 + k == me ? make_float2(m, l) : __ldcg(&p.stat[share_at(g, k) * p.slot_rows + t * kTile + r]);
                        top = fmaxf(top, st[k].x);
                    }
                    const float ref = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < kDirect; ++k) {
                        weight[k] = ex2(st[k].x - ref);
                        sum = fmaf(st[k].y, weight[k], sum);
                    }
                    m = top;
                    l = sum;
                    if (lane == 0) *of_unit = 0;
                }
            }
            if (any) {
                const float inv = 1.f / l;
                const int64_t out_row = real ? attend_out_row(p, a, rt) : 0;
                const bool dirty = *static_cast<volatile int *>(&b.dirty);
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    __syncwarp();
                    float o[32];
                    if (cnt > 0) {
                        tmem_ld32(co + d, o);
                        if (take) {
                            float y[32];
                            tmem_ld32(co + 128 + d, y);
                            tmem_ld_wait();
                            reg_fence(o);
                            reg_fence(y);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = fmaf(o[j], w_mine, y[j] * w_other);
                        } else {
                            tmem_ld_wait();
                            reg_fence(o);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0.f;
                    }
                    if (!real) continue;
                    if (dirty) {   // what was taken out of V, for rows that see it
                        const int k1 = min(sees, (g.first + g.n) * kTile);
                        for (int k = max(from, g.first * kTile); k < k1; ++k) {
                            const int page = p.table[(int64_t)a.list * p.max_pages + (k >> p.shift)];
                            if (page < 0 || page >= p.n_pages) continue;
                            if constexpr (BITS != 0) {   // the group of these channels
                                const QuantRow row = quant_row(BITS, 2 * KH, ((int64_t)page << p.shift) + (k & ((1 << p.shift) - 1)));
                                const uint16_t word = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p.v_pool) + row.words)[d / 32];
                                if (quant_is_nan<BITS>(word)) {
#pragma unroll
                                    for (int j = 0; j < 32; ++j) o[j] = NAN;
                                }
                                continue;
                            }
                            const uint16_t *vr = static_cast<const uint16_t *>(p.v_pool) +
                                (((int64_t)page << p.shift) + (k & ((1 << p.shift) - 1))) * D + d;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const uint32_t bits = vr[j];
                                if ((bits & 0x7f80u) == 0x7f80u) o[j] += __uint_as_float(bits << 16);
                            }
                        }
                    }
                    if (direct) {
                        float sum[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[j] = 0.f;
#pragma unroll
                        for (int k = 0; k < kDirect; ++k) {
                            if (k >= n) break;
                            if (g.c0 + k == me) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) sum[j] = fmaf(o[j], weight[k], sum[j]);
                            } else {
                                const float *src = p.part + (share_at(g, k) * p.slot_rows + t * kTile + r) * D + d;
#pragma unroll
                                for (int j = 0; j < 32; j += 8) {
                                    float y[8];
                                    load8(src + j, y);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) sum[j + e] = fmaf(y[e], weight[k], sum[j + e]);
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = sum[j];
                    }
                    if (g.whole || direct) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + out_row * D + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t q[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // a row that sees nothing: zeros, whatever O holds
                                const float y0 = sees > 0 ? o[8 * j + 2 * e] * inv : 0.f;
                                const float y1 = sees > 0 ? o[8 * j + 2 * e + 1] * inv : 0.f;
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q[e]) : "f"(y1), "f"(y0));
                            }
                            dst[j] = make_uint4(q[0], q[1], q[2], q[3]);
                        }
                    } else {
                        float *dst = p.part + slot * D + d;
#pragma unroll
                        for (int j = 0; j < 32; j += 8) store8(dst + j, o + j);
                    }
                }
                if (real) {
                    if (g.whole || direct)
                        attend_store_lse(p, out_row, m, l, sees > 0);
                    else
                        p.stat[slot] = make_float2(m, l);
                }
            }
            __syncwarp();
            tc_fence_before();   // O is read: the next unit's products may overwrite it
            if (take && lane == 0) mbar_arrive(&b.half_empty);
            if (!g.whole) {
                // the CTA that finishes last joins the unit's slots
                const int c0 = g.c0, c1 = g.c1;
                const int groups = attend_groups(n);
                const int g0 = c0 + (me - c0) / kJoinGroup * kJoinGroup, gn = min(kJoinGroup, c1 - g0 + 1);
                const AttendSpan group{c0, g0, 1, gn, false, false};
                const AttendSpan unit{c0, c0, groups > 1 ? kJoinGroup : 1, groups > 1 ? groups : n, groups > 1, true};
                uint32_t *of_group = &p.arrived[16 * g0 + 8 + 4 * t + (rows > 32 ? quarter : 0)];
                if (rows > 32) {   // each warp its own 32 rows
                    const int row0 = 32 * quarter, mine = min(32, rows - row0);
                    bool last = any && !direct;
                    if (last && groups > 1) {
                        last = attend_last(of_group, gn);
                        if (last)
                            attend_join<__nv_bfloat16, 4, 4>(p, a, group, t * R + row0, mine, t * kTile + row0, lane, 32);
                    }
                    if (last && attend_last(of_unit, unit.n))
                        attend_join<__nv_bfloat16, 4, 4>(p, a, unit, t * R + row0, mine, t * kTile + row0, lane, 32);
                } else {           // one warp's rows: often of many slots, so all four join
                    // the first warp counts and tells the others
                    auto all_last = [&](uint32_t *count, int of, bool *is) {
                        volatile int *last = &b.last[t][nwg & 1];
                        if (quarter == 0) {
                            const bool x = attend_last(count, of);
                            if (lane == 0) {
                                *last = x;
                                mbar_arrive(&b.wg[t]);
                            }
                        }
                        if (!warp_wait(&b.wg[t], nwg++ & 1, stop, p.status)) return false;
                        *is = *last;
                        return true;
                    };
                    bool last = true;
                    if (groups > 1) {
                        if (!(ok = all_last(of_group, gn, &last))) break;
                        if (last) {
                            attend_join<__nv_bfloat16, 2, 4>(p, a, group, t * R, rows, t * kTile, r, kTile);
                            __threadfence();   // before the first warp counts for all four
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&b.joined[t]);
                            if (!(ok = warp_wait(&b.joined[t], njoined++ & 1, stop, p.status))) break;
                        }
                    }
                    if (last) {
                        if (!(ok = all_last(of_unit, unit.n, &last))) break;
                        if (last) attend_join<__nv_bfloat16, 2, 4>(p, a, unit, t * R, rows, t * kTile, r, kTile);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// bf16 q as [token][KV head][query head][D] in 128-byte swizzled boxes of 64 x box
// elements (make_tma_map has three dimensions, of contiguous rows).
bool make_q_map(CUtensorMap *m, const void *q, const uint64_t (&dims)[4], const uint64_t (&strides)[3],
                const uint32_t (&box)[4]) {
    static std::atomic<void *> entry{nullptr};
    void *fn = entry.load(std::memory_order_relaxed);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            return false;
        entry.store(fn, std::memory_order_relaxed);
    }
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, steps,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KH, bool TWO, int BITS>
int launch(AttendParams &p, int grid, cudaStream_t st) {
    const uint64_t D = 64 * KH, G = p.group;
    const uint32_t tokens = kTile / p.group;
    CUtensorMap tq, tk{}, tv{};   // held rows have no use for the last two
    const uint64_t dims[4] = {D, G, (uint64_t)p.n_kv_heads, (uint64_t)p.n_tokens};
    const uint64_t strides[3] = {D * 2, G * D * 2, (uint64_t)p.q_stride * 2};
    const uint32_t box[4] = {64, (uint32_t)G, 1, tokens};
    const uint64_t ps = (uint64_t)1 << p.shift;
    if (!make_q_map(&tq, p.q, dims, strides, box) ||
        (BITS == 0 && (!make_tma_map(&tk, p.k_pool, D, ps, (uint64_t)p.n_pages, (uint32_t)ps) ||
                       !make_tma_map(&tv, p.v_pool, D, ps, (uint64_t)p.n_pages, (uint32_t)ps)))) {
        set_error("%s: cuTensorMapEncodeTiled failed (alignment or driver)", attend_name(p));
        return KVC_ERR_CUDA;
    }
    constexpr size_t bytes = smem_bytes<KH, BITS>();
    static_assert(bytes <= 232448, "shared memory of one block");
    static AskedOnce asked;
    cudaError_t err = cudaSuccess;
    const int regs = asked.get([&] {
        cudaFuncAttributes at{};
        err = cudaFuncGetAttributes(&at, attend_tc_kernel<KH, TWO, BITS>);
        return err == cudaSuccess ? at.numRegs : 0;
    });
    if (err != cudaSuccess) {
        cudaGetLastError();
        set_error("%s: the tensor-core kernel's attributes: %s", attend_name(p), cudaGetErrorString(err));
        return KVC_ERR_CUDA;
    }
    // (of a library built by the compiler it was measured with, these are 168 or 96)
    if (regs != Shape<BITS>::kRegsLaunch) {
        set_error("%s: the tensor-core kernel has %d registers per thread, its split needs %d", attend_name(p), regs,
                  Shape<BITS>::kRegsLaunch);
        return KVC_ERR_UNSUPPORTED;
    }
    allow_shared<attend_tc_kernel<KH, TWO, BITS>>((int)bytes);
    launch_early(attend_tc_kernel<KH, TWO, BITS>, grid, Shape<BITS>::kThreads, bytes, st, tq, tk, tv, p);
    return cache_launched(attend_name(p));
}

// The units' shape for lists of more than rows_above rows; false if there are too many.
bool shape_units(AttendParams &p, int rows_above) {
    const char *skip = getenv("KVC_TEST_SKIP_ARRIVE");
    p.skip_load = skip && skip[0] == '1';
    const int R = kTile / p.group * p.group;   // whole tokens
    p.split_rows = R;
    p.step_keys = kTile;
    p.extra = p.bits != 0 && p.dim == 128 ? kExtraHeld : kExtra;
    if (attend_units(p, 2 * R, rows_above, INT_MAX)) return true;
    set_error("%s: n_seqs * n_kv_heads * max_new is too large", attend_name(p));
    return false;
}

}  // namespace

}  // namespace kvc
