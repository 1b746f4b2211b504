// chunk_tc.cu -- the prefill attention calls on the sm_103a tensor cores, for
// 16-bit queries of head dim 64 or 128 over a BF16 or FP8-E4M3 paged cache.
//
// A CTA works through units of the plan (chunk_plan.cuh): two tiles of 128
// query rows (128 / G tokens with their G heads each) of one kv head, over a
// piece of their key blocks.  A page of 128 keys is in shared memory once for
// both tiles; each tile takes it in two steps of 64 keys:
//
//   S_i  = Q_i K^T       tcgen05.mma, M = 128 rows, N = 64 keys, into one of
//                        the tile's two tensor-memory buffers
//   P_i  = 2^(S_i c - m) one thread per row; its 64 logits sit in registers and
//                        their maximum comes with the tensor-memory load, so
//                        neither needs an exchange
//   O_i += P_i V         kind::f16, P from tensor memory (written over its own
//                        S), V as it lies in the page (MN-major)
//
// Each tile has a warp that issues its products, in the order P V(k), Q K^T(k +
// 2) into the buffer that P(k) leaves: a step's logits are there when the last
// step's softmax ends, and one tile's softmax runs while the other's products
// do.  Products of one issuing thread run in the order they are issued: S(k +
// 2) is written after P V(k) has read P(k) from the same columns.  A commit
// covers everything issued before it, so whoever sees S(k + 2) knows that
// P V(k) is done.
//
// BF16 pages are multiplied as they are.  E4M3 keys are too, against two E4M3
// terms of each bf16 query (kind::f8f6f4), and E4M3 values are widened to f16
// (exact) by a warpgroup of their own; f16 queries, and heads of 64 dims, have
// their keys widened as well.
//
// Softmax: c = sm_scale * k_scale * log2(e) > 0.  The exponent offset m of a
// row is raised only when a step's maximum, as a power of two, exceeds it by
// more than kRaise (then the row's O is rescaled in tensor memory), so p <=
// 2^kRaise, times 2^7 where P is f16.  It is rounded to the 16-bit type of the products (off by at
// most 2^-8 of itself in bf16, of either sign, so an output of many keys keeps
// about the bf16 rounding of its own); the row sum takes it unrounded, in fp32.
//
// A tile takes the pages that its own query blocks list (every page without a
// selection), and passes the other tile's by; only rows of different query
// blocks within a tile test their own bitmaps.  A pair of one tile of rows (a
// short chunk, or the end of one) is worked on by both tiles all the same: each
// holds the rows, takes every other page and keeps sums of its own, and the
// first tile joins them at the end (the second one's O lies in the same
// tensor-memory lanes).
//
// Keys that a row does not read take p = 0 by its limit, a count of keys.  A
// product with V would still turn 0 * NaN into NaN, so the V page of a block
// that some row does not read in full is scrubbed in shared memory first: keys
// that no row reads become zeros, and elements that are not finite become zeros
// and leave a mark; rows that do read such a key look its elements up in the
// page at the end and take the NaN or infinity from there.
//
// What bounds it: the tensor pipe needs 64 cycles for 128 x 128 x 16, 2048 a
// page and two tiles, but shared memory delivers the operands of N = 64 steps
// in 48 instead of 32 cycles: 2560.  The exponentials of the page take 1024 on
// the special-function units of an SM, the softmax of one step about 1000 from
// logits to P.  Beside the pipe it is the fetching of instructions: sixteen
// warps run a dozen roles' code, so waits, steps and epilogues are kept short
// (where each measured, it is said there).  Measured (eight 512-token chunks at
// up to 15872 cached tokens, 64 / 8 heads of 128 dims, a graph of calls on one
// set of inputs; called one by one on changing ones in brackets): 466 (500) us
// over BF16, 1.54 (1.43) PFLOP/s, 80 (75) % of the measured bf16 rate; the same
// chunks over 32 selected E4M3 blocks a query block 346 (355) us, 1.30 (1.26)
// PFLOP/s.  Steps of 128 keys with one buffer a tile, where the next product
// waits for the whole softmax, took 7 % more.  A short chunk (16 tokens of four
// requests over 14000 keys, 57 (61) us, 18 of HBM time) is 24 us of products,
// its 128 rows against two E4M3 terms; the others are the plan, the first unit's
// records, page list and queries (10), and the join (6).  Where neighbouring
// tiles select different pages (query blocks of 16 tokens over BF16, 60 to 64
// (69) us) it waits for the L2: 64 KB a page for one tile, 590 MB in all, two
// pages of each kind in flight.
//
// Roles (16 warps): warps 0-3 and 4-7 the softmax and epilogue of tile 0 and 1
// (warp w reads TMEM lanes 32 (w % 4) .. +31), warps 8-11 split queries, widen
// and scrub, warp 12 issues the TMA loads, warps 13 and 15 the products of tile
// 0 and 1 (warp 13 owns tensor memory), warp 14 claims units and builds their
// page lists one unit ahead.  Every wait is bounded: one that gives up sets bit
// 0 of the workspace status word and the CTA winds down.
#include <limits.h>
#include <math.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "block_scale.cuh"
#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace spd {

namespace {

constexpr int kRows = 128;           // query rows of a tile (M)
constexpr int kKeys = kBlock;        // keys of a page
constexpr int kHalf = kKeys / 2;     // keys of a step (N of S, K of P V)
constexpr int kThreads = 512;
constexpr int kWarpSide = 8, kWarpTma = 12, kWarpMma = 13, kWarpSched = 14, kWarpMma1 = 15;
constexpr int kBox = 128 * 128;      // 64 dims of 128 rows of a 16-bit type, bytes
constexpr float kRaise = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
// registers: 128 a thread at launch; the softmax warpgroups rise to 152, the
// two others drop to 104
constexpr uint32_t kRegsSoft = 152, kRegsOther = 104;
static_assert(256 * kRegsSoft + 256 * kRegsOther <= kThreads * 128, "register split");
constexpr uint32_t kUnitReleases = 8 + 4 + 1 + 2;  // warps that read a unit record
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;         // S_i at 128 i (two buffers of 64), O_i at 256 + 128 i

// How a cache is multiplied.
enum Mode {
    kModeBf16,   // BF16 pages as they are, bf16 queries
    kModeTerms,  // E4M3: K as it is against two E4M3 terms of each bf16 query, V widened to f16
    kModeWide    // E4M3: K and V widened to f16, f16 queries (bf16 ones made f16)
};

template <int D, Mode M>
struct Shape {
    static constexpr bool kF8 = M != kModeBf16;
    static constexpr int kBoxes = D / 64;
    static constexpr int kTileQ = kBoxes * kBox;  // one tile of queries
    static constexpr int kPage16 = kBoxes * kBox; // a K or V page of 16-bit elements
    static constexpr int kPage8 = kKeys * D;      // one of E4M3
    // K pages as the products read them, V pages likewise, and E4M3 pages that wait to be widened
    static constexpr int kPageK = M == kModeTerms ? kPage8 : kPage16;
    static constexpr int kKs = M == kModeBf16 ? 2 : (M == kModeTerms ? 3 : 1);
    static constexpr int kVs = 2;
    static constexpr int kRs = M == kModeBf16 ? 0 : (M == kModeTerms ? 2 : 3);
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kTileQ;
    static constexpr int kOffV = kOffK + kKs * kPageK;
    static constexpr int kOffRaw = kOffV + kVs * kPage16;
    static constexpr int kEnd = kOffRaw + kRs * kPage8;
};

// A place in a ring of N slots, and the parity of its present round.
template <int N>
struct Ring {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            ++round;
        }
    }
    __device__ __forceinline__ uint32_t parity() const { return round & 1; }
};

// Pages of scales (block-scaled caches).  While a tile's softmax is on a page,
// its products have taken or passed at most the next one, and three K pages at
// most wait behind that: the loader is four pages ahead at most.
constexpr int kScaleRing = 8;

constexpr int kTakeShift = 14;
constexpr uint32_t kBlockMask = (1u << kTakeShift) - 1;

struct UnitRec {
    int32_t nblk;        // key blocks; -1: no more units
    int32_t tok0, i0, nt;  // first query token, its index in the chunk, tokens
    int32_t h, tiles;    // kv head; tiles at work
    int32_t dual;        // one tile of rows: both tiles hold them and take every other page
    int32_t own[2];      // pages that each tile takes
    int32_t pre, cap;    // a row's limit is min(pre + i + 1, cap), at least 0
    int32_t lim_lo;      // limits of the first and the last token
    int32_t lim_hi;
    int32_t mixed;       // bit per tile: rows of several query blocks, each tests its own bitmap
    int32_t qrow0, qrow_end;  // selection row of the sequence's first token, and the end of its rows
    int32_t pieces, part;     // pieces of the pair; partial slot of this one
    int32_t marked;      // some V element of a scrubbed block is not finite
    int32_t page[kMaxNB];
    uint16_t kb[kMaxNB];  // key block, and from kTakeShift on a bit per tile that takes it
    uint32_t marks[kMaxNB / 32];  // key blocks that hold such elements
};

struct Shared {
    uint64_t u_full[2], u_empty[2];
    uint64_t q_full, q_empty, q_ready[2][2];  // ready: by parity of the units with products, and tile
    uint64_t k_full[3], k_empty[3];           // K pages for the products
    uint64_t v_full[2], v_ready[2], v_empty[2];  // V pages: loaded (BF16), widened or scrubbed, read
    uint64_t r_full[3], r_empty[3];           // E4M3 pages to be widened
    uint64_t s_full[2][2], p_full[2][2];      // by tile and half of a page's keys
    uint64_t pv_done[2];                      // by tile: the product of one more half is done
    uint64_t o_full[2], o_free[2];
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    uint64_t dual_ready;              // the second tile's sums of a dual unit
    float2 dual_stats[kRows];         // its rows' exponent offsets and sums
    float2 scale[kScaleRing];         // scales of a page, by page ordinal
    float row_factor[2][2 * kRows];  // by parity of the units with products: what the queries' scaling takes from the logits
    UnitRec unit[2];
};

struct TcArgs {
    ChunkArgs a;
    ChunkLayout lay;
    char *ws;
    int32_t G, heads_built, q_f16;
    float c;  // sm_scale * k_scale * log2(e)
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same, and the largest of the 32 values (a NaN among them is passed over).
__device__ __forceinline__ float tmem_ld32_max(uint32_t taddr, float *v) {
    uint32_t r[32], top;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(top)
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
    return __uint_as_float(top);
}

// Waits for the loads issued so far; the 33 registers of one of them pass
// through, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld32(float *v, float &top) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31]), "+f"(top)
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Matrix descriptors of the 128-byte-swizzled operands (128 rows or keys of
// 128 bytes, 8-row groups 1024 bytes apart; `lbo`: the next 64 dims of an
// MN-major operand).  Only the address field differs between the steps of a
// product, so a product builds the low word once and each step adds a
// constant to it.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (static_cast<uint32_t>(tc::kSw128) << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// D (+)= A B, A and B in shared memory: kind::f16, or kind::f8f6f4 (E4M3).
template <bool kF8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t add) {
    if (kF8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "mov.b64 a, {%1, %4};\n\t"
            "mov.b64 b, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(kDescHigh), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "mov.b64 a, {%1, %4};\n\t"
            "mov.b64 b, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(kDescHigh), "r"(add)
            : "memory");
}

// D (+)= A B, kind::f16, A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_low), "r"(idesc), "r"(kDescHigh), "r"(add)
        : "memory");
}

// 32 bytes, a whole memory sector, in one store (32-byte aligned).
__device__ __forceinline__ void store32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// One lane of the converged warp, the same one every time.  It is asked anew
// for every product: from its answer the compiler knows that one thread issues
// the products.  (A loop-invariant answer kept in a variable must not be used
// instead: it invites the compiler to give the two kinds of lanes loops of
// their own, which then run interleaved.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one)::"memory");
    return one != 0;
}

__device__ __forceinline__ bool aborted(Shared &sh) { return *reinterpret_cast<volatile int *>(&sh.abort) != 0; }

__device__ __forceinline__ bool wait_or_abort(Shared &sh, uint64_t *bar, uint32_t parity) {
    if (tc::mbar_wait_tries(bar, parity)) return true;
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
    return false;
}

// Warp-uniform wait, for the warp-collective accesses that follow it.
__device__ __forceinline__ bool warp_wait(Shared &sh, uint64_t *bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_tries(bar, parity));
    if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
    return ok;
}

// Arrival of a whole warp, after what its lanes wrote.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    return tc::f32x2_to_f16x2(lo, hi);
}

__device__ __forceinline__ int32_t row_limit(const UnitRec &u, int32_t i) {
    return max(min(u.pre + i + 1, u.cap), 0);
}

__device__ __forceinline__ bool finite_bits(uint32_t x, bool bf16) {
    const uint32_t e = bf16 ? 0x7f80u : 0x7c00u;
    return (x & e) != e;
}

// The largest magnitude of one bf16 query row of D dims in its swizzled tile,
// as the power of two that brings it to [2^top, 2^(top + 1)), and the inverse.
// A row with an infinity or a NaN is multiplied by NaN: its logits are infinite
// or NaN, so no softmax of it is finite, and E4M3 has no infinity to hold.
template <int D>
__device__ __forceinline__ void row_power(const uint8_t *q, int row, int top, float &up, float &down) {
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
            const uint4 w = *reinterpret_cast<const uint4 *>(q + b * kBox + ((ch ^ (row & 7)) << 4));
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
    const int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7);  // biased exponent
    const int shift = e == 0 ? 0 : min(top - (e - 127), 100);
    up = e == 255 ? NAN : __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
    down = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
}

// A bf16 query row to f16, in place, scaled by a power of two into [2^14,
// 2^15): exact for elements within 2^31 of the row's largest (eight bits above
// f16's smallest step of 2^-24), and off by at most 2^-39 of that beyond.
// Returns the inverse scale.
template <int D>
__device__ __forceinline__ float halve_query_row(uint8_t *q, int row) {
    float up, down;
    row_power<D>(q, row, 14, up, down);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
#pragma unroll 2
        for (int ch = 0; ch < 8; ++ch) {
            uint4 *at = reinterpret_cast<uint4 *>(q + b * kBox + ((ch ^ (row & 7)) << 4));
            uint4 w = *at;
            uint32_t *wp = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wp[i] = tc::f32x2_to_f16x2(__uint_as_float(wp[i] << 16) * up, __uint_as_float(wp[i] & 0xffff0000u) * up);
            *at = w;
        }
    return down;
}

// A bf16 query row of 128 dims as two E4M3 terms, in place: the row is scaled
// by a power of two into [128, 256); the first term is its rounding to four
// bits, the second what is left (four more bits: the sum is exact for elements
// within 2^9 of the row's largest, and off by at most 2^-17 of that beyond).
// 32 dims, one step of the product, take 64 bytes as bf16: their first terms
// go into the first 32 of these, their second terms into the others, so no
// group waits for another.  Returns the inverse scale.
__device__ __forceinline__ float split_query_row(uint8_t *q, int row) {
    float up, down;
    row_power<128>(q, row, 7, up, down);
    const uint64_t up2 = pair(up, up);
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
        uint8_t *box = q + (g >> 1) * kBox;
        uint32_t t0[8], t1[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 w = *reinterpret_cast<const uint4 *>(box + ((((g & 1) * 4 + c) ^ (row & 7)) << 4));
            const uint32_t wp[4] = {w.x, w.y, w.z, w.w};
            uint32_t a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                unpair(mul2(pair(__uint_as_float(wp[i] << 16), __uint_as_float(wp[i] & 0xffff0000u)), up2), lo, hi);
                const __half2 h = __floats2half2_rn(lo, hi);  // eight bits of a value below 256: exact
                a[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
                const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(a[i]), __NV_E4M3);
                b[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(h, __half2(back))), __NV_SATFINITE,
                                                  __NV_E4M3);
            }
            t0[2 * c] = a[0] | (a[1] << 16);
            t0[2 * c + 1] = a[2] | (a[3] << 16);
            t1[2 * c] = b[0] | (b[1] << 16);
            t1[2 * c + 1] = b[2] | (b[3] << 16);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            *reinterpret_cast<uint4 *>(box + ((((g & 1) * 4 + c) ^ (row & 7)) << 4)) =
                make_uint4(t0[4 * c], t0[4 * c + 1], t0[4 * c + 2], t0[4 * c + 3]);
            *reinterpret_cast<uint4 *>(box + ((((g & 1) * 4 + 2 + c) ^ (row & 7)) << 4)) =
                make_uint4(t1[4 * c], t1[4 * c + 1], t1[4 * c + 2], t1[4 * c + 3]);
        }
    }
    return down;
}

// Elements of the marked blocks' V rows that this row reads (keys below lim, of
// its own selection where row_bits is given) and that are not finite, added to
// the row's O in tensor memory, where the products saw zeros in their place.
// The two sums of a dual unit are joined first, with their weights, and the
// second one left zero: an infinity of one tile's page is not to meet the other
// tile's weight, which may be 0.  A warp-collective, and a rare, call.
template <int D, bool F8>
__device__ __noinline__ void take_marked(const TcArgs &t, const UnitRec &u, int tile, int32_t lim,
                                         const uint32_t *row_bits, uint32_t col_o, float w_own, float w_other) {
    const ChunkArgs &a = t.a;
    uint32_t odd[3][D / 32];  // NaN, +inf, -inf dims
    for (int k = 0; k < 3; ++k)
        for (int i = 0; i < D / 32; ++i) odd[k][i] = 0;
    uint32_t all = 0;  // all dims NaN: nothing more to find
    for (int at = 0; at < u.nblk && all != 0xffffffffu; ++at) {
        const uint32_t entry = u.kb[at];
        const int kb = entry & kBlockMask;
        if (kb * kKeys >= lim || !((u.marks[kb >> 5] >> (kb & 31)) & 1u)) continue;
        if (!u.dual && !((entry >> (kTakeShift + tile)) & 1u)) continue;  // only the other tile's rows read it
        if (row_bits != nullptr && !((row_bits[kb >> 5] >> (kb & 31)) & 1u)) continue;
        const int64_t page = u.page[at];
        const int n = min(kKeys, lim - kb * kKeys);
        for (int i = 0; i < n && all != 0xffffffffu; ++i) {
            const uint8_t *v = a.v + ((page * kKeys + i) * a.v_s0 + u.h * a.v_s1) * (F8 ? 1 : 2);
            for (int d0 = 0; d0 < D; d0 += F8 ? 16 : 8) {
                const uint4 w = *reinterpret_cast<const uint4 *>(v + d0 * (F8 ? 1 : 2));
                const uint32_t wp[4] = {w.x, w.y, w.z, w.w};
                for (int k = 0; k < 4; ++k) {
                    if (F8 ? __vcmpeq4(wp[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) == 0
                           : finite_bits(wp[k], true) && finite_bits(wp[k] >> 16, true))
                        continue;
                    for (int e = 0; e < (F8 ? 4 : 2); ++e) {
                        const int d = d0 + k * (F8 ? 4 : 2) + e;
                        const uint32_t x = F8 ? (wp[k] >> (8 * e)) & 0xffu : (wp[k] >> (16 * e)) & 0xffffu;
                        if (F8 ? (x & 0x7fu) == 0x7fu : (x & 0x7fffu) > 0x7f80u) odd[0][d >> 5] |= 1u << (d & 31);
                        else if (!F8 && (x & 0x7fffu) == 0x7f80u) odd[x >> 15 ? 2 : 1][d >> 5] |= 1u << (d & 31);
                    }
                }
            }
            all = 0xffffffffu;
            for (int k = 0; k < D / 32; ++k) all &= odd[0][k];
        }
    }
    __syncwarp();
    for (int c0 = 0; c0 < D; c0 += 16) {
        float o[16];
        tc::tmem_ld16(col_o + c0, o);
        tc::tmem_wait_ld();
        if (u.dual) {
            float x[16];
            tc::tmem_ld16(col_o + 128 + c0, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i] = fmaf(o[i], w_own, x[i] * w_other);
                x[i] = 0.f;
            }
            tc::tmem_st16(col_o + 128 + c0, x);
        }
        const uint32_t nan = odd[0][c0 >> 5] >> (c0 & 31), pos = odd[1][c0 >> 5] >> (c0 & 31),
                       neg = odd[2][c0 >> 5] >> (c0 & 31);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if ((nan >> i) & 1u) o[i] = NAN;
            if ((pos >> i) & 1u) o[i] += INFINITY;
            if ((neg >> i) & 1u) o[i] -= INFINITY;
        }
        tc::tmem_st16(col_o + c0, o);
        tc::tmem_wait_st();
    }
}

// What half a page of a low V scale (block_scale.cuh) adds to a row's sum: 2^(z + off)
// of its first `left` keys.  Rare, so short and out of line: over the logits in
// registers, unrolled, it cost every page 2 % in instructions to fetch.
__device__ __noinline__ float low_page_sum(uint32_t col, int left, float c, float off) {
    float l = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < kHalf; i0 += 8) {
        float z[8];
        tc::tmem_ld8(col + i0, z);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) l += i0 + i < left ? tc::ex2(fmaf(z[i], c, off)) : 0.f;
    }
    return l;
}

// kBs: block-scaled caches (block_scale.cuh); E4M3 modes only.
template <int D, Mode M, bool kBs>
__global__ void __launch_bounds__(kThreads, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TcArgs t) {
    using S = Shape<D, M>;
    constexpr bool F8 = S::kF8, kBf16 = !F8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared &sh = *reinterpret_cast<Shared *>(smem + S::kEnd);
    const ChunkArgs &a = t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ChunkHeader *hd = reinterpret_cast<ChunkHeader *>(t.ws + t.lay.header);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.u_full[i], 1);
            tc::mbar_init(&sh.u_empty[i], kUnitReleases);
            tc::mbar_init(&sh.o_full[i], 1);
            tc::mbar_init(&sh.pv_done[i], 1);
            tc::mbar_init(&sh.o_free[i], 4);
            for (int k = 0; k < 2; ++k) {
                tc::mbar_init(&sh.q_ready[i][k], 4);
                tc::mbar_init(&sh.s_full[i][k], 1);
                tc::mbar_init(&sh.p_full[i][k], 4);
            }
            tc::mbar_init(&sh.v_full[i], 1);
            tc::mbar_init(&sh.v_ready[i], 4);
            tc::mbar_init(&sh.v_empty[i], 2);
        }
        for (int i = 0; i < 3; ++i) {
            // its widening warps, or the copy (and the scales')
            tc::mbar_init(&sh.k_full[i], M == kModeWide ? 4 : (kBs ? 2 : 1));
            tc::mbar_init(&sh.k_empty[i], 2);
            tc::mbar_init(&sh.r_full[i], M == kModeWide && kBs ? 2 : 1);
            tc::mbar_init(&sh.r_empty[i], 4);
        }
        tc::mbar_init(&sh.dual_ready, 4);
        tc::mbar_init(&sh.q_full, 1);
        tc::mbar_init(&sh.q_empty, 2);
        tc::mbar_init(&sh.drain[0], 1);
        tc::mbar_init(&sh.drain[1], 1);
        sh.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kWarpMma) tc::tmem_alloc(&sh.tmem_base, kTmemCols);
    if (threadIdx.x == kWarpTma * 32) {
        tc::prefetch_tmap(&tmap_q);
        tc::prefetch_tmap(&tmap_k);
        tc::prefetch_tmap(&tmap_v);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    tc::pdl_wait();  // the plan
    tc::pdl_trigger();

    if (warp < kWarpSide) {
        tc::regs_inc<kRegsSoft>();
        // ----------------------------------------------- softmax, epilogue
        const int tile = warp >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t col_s = tmem + lane_base + kColS + tile * 128;
        const uint32_t col_o = tmem + lane_base + kColO + tile * 128;
        const int tile_tok = r / t.G, g = r % t.G;  // token within the tile, head within the group
        const bool in_tile = r < t.lay.tt * t.G;
        uint32_t n_s = 0, n_o = 0;  // S buffers seen, O tiles seen
        uint32_t nq = 0, n_dual = 0;  // units with products, dual units
        uint32_t n_pages = 0;         // pages of the units so far
        for (uint32_t n = 0;; ++n) {
            UnitRec &u = sh.unit[n & 1];
            if (!warp_wait(sh, &sh.u_full[n & 1], (n >> 1) & 1) || u.nblk < 0) break;
            const int nblk = u.nblk;
            const bool dual = u.dual != 0;
            const int j_tok = tile_tok + (dual ? 0 : tile * t.lay.tt);  // token within the pair
            const bool have = in_tile && j_tok < u.nt;
            const int32_t lim = have ? row_limit(u, u.i0 + j_tok) : 0;
            const uint32_t iq = nq, page0 = n_pages;
            if (nblk > 0) ++nq;
            n_pages += nblk;
            if (tile >= u.tiles) {
                warp_arrive(&sh.u_empty[n & 1], lane);
                continue;
            }
            const uint32_t *bits = nullptr;  // the row's own selection, when the unit's rows differ
            bool chosen = true;
            const bool mixed = (u.mixed >> tile) & 1;
            const int own = u.own[tile];
            if (mixed && have) {
                const int64_t row = static_cast<int64_t>(u.qrow0) + (u.i0 + j_tok) / a.bsq;
                chosen = row >= 0 && row < u.qrow_end;
                if (chosen)
                    bits = reinterpret_cast<const uint32_t *>(t.ws + t.lay.bitmaps) +
                           ((t.heads_built > 1 ? static_cast<int64_t>(u.h) : 0) * a.n_rows + row) * t.lay.words;
            }
            float c = t.c;
            if (F8 && own > 0) {
                if (!warp_wait(sh, &sh.q_ready[iq & 1][tile], (iq >> 1) & 1)) break;
                c *= sh.row_factor[iq & 1][tile * kRows + r];
            }
            float m_run = -INFINITY, l = 0.f;
            float threshold = -INFINITY;  // logits above it raise the offset
            // f16 P starts at 2^7, so that small weights stay normal numbers
            // down to 2^-21 of the largest (and 2^kRaise more fits below 65504)
            constexpr float kLift = kBf16 ? 0.f : 7.f;
            uint64_t c2 = pair(c, c);
            uint64_t m2 = 0;              // minus the offset, twice (0 while the row has none)
            // block-scaled: the page's logit factor and its V scale; the threshold
            // is in log2 units then, m2 without the V scale
            float cb = c;
            BlockScale bs = {1.f, 0.f, 1.f};
            int look = kHalf;             // rows with fewer keys left are looked at more closely: all of a low page's
            bool seen = false, ok = true;
            int word_at = -1;
            uint32_t word = 0;
            // Half a page, 64 keys, is a step of the online softmax.  Its logits
            // lie in one of two buffers, and its P goes over them.
            // (Two copies of a step cost the fetching of their instructions, one
            // costs the addresses: dense bf16 465 us with two, 486 with one, over
            // E4M3, where the queries' terms and the widening want the
            // instruction cache too, ragged 98 and 95, drawn small batches 2 %.)
            constexpr int kUnrolled = kBf16 ? 2 : 1;
            for (int j = 0, done = 0; done < own && ok; ++j) {
                const uint32_t entry = u.kb[j];
                if (!((entry >> (kTakeShift + tile)) & 1u)) continue;  // the other tile's page
                const int kb = entry & kBlockMask;
                int left = lim - kb * kKeys;  // keys of the page that the row reads
                if (mixed) {
                    if (bits != nullptr && (kb >> 5) != word_at) {
                        word_at = kb >> 5;
                        word = bits[word_at];
                    }
                    if (!chosen || !((word >> (kb & 31)) & 1u)) left = 0;
                }
                seen |= left > 0;
                const bool partial = mixed || (kb + 1) * kKeys > u.lim_lo;  // some row does not read it all
#pragma unroll kUnrolled
                for (int h = 0; h < 2; ++h) {
                    ok = warp_wait(sh, &sh.s_full[tile][h], n_s & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                    if (kBs && h == 0) {
                        bs = block_scale(sh.scale[(page0 + j) % kScaleRing]);
                        look = low_scale(bs) ? INT_MAX : kHalf;
                        cb = fmaxf(c * bs.k, 1e-37f);  // above 0: masked logits are -inf
                        c2 = pair(cb, cb);
                    }
                    float x[kHalf], top[2];
                    top[0] = tmem_ld32_max(col_s + h * kHalf, x);
                    top[1] = tmem_ld32_max(col_s + h * kHalf + 32, x + 32);
                    if (h == 1) left -= kHalf;
                    tmem_wait_ld32(x, top[0]);
                    tmem_wait_ld32(x + 32, top[1]);
                    uint64_t sum[2] = {0, 0};
                    if (partial && __all_sync(0xffffffffu, left <= 0)) {
                        // none of the warp's rows reads these keys (another
                        // query block's selection, or keys behind the first
                        // tile): P = 0
                        uint32_t zero[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch) tmem_st16u(col_s + h * kHalf + ch * 16, zero);
                    } else {
                        float mx = fmaxf(top[0], top[1]);
                        if (kBs) mx = fmaf(mx, cb, bs.lg_v);
                        if (__any_sync(0xffffffffu, left < look || mx > threshold)) {
                            if (left < kHalf) {
                                mx = -INFINITY;
#pragma unroll
                                for (int i = 0; i < kHalf; ++i) {
                                    x[i] = i < left ? x[i] : -INFINITY;
                                    mx = fmaxf(mx, x[i]);
                                }
                                if (kBs) mx = fmaf(mx, cb, bs.lg_v);
                            }
                            // raise the offset if the step's maximum runs more
                            // than 2^kRaise above it (or the row had none yet)
                            const bool raise = mx > threshold;
                            float alpha = 1.f;
                            if (raise) {
                                const float bm = kBs ? mx - kLift : fmaf(mx, c, -kLift);
                                alpha = kBs ? rescale(l, m_run - bm) : tc::ex2(m_run - bm);  // 0 for a row that had none
                                if (!kBs) l *= alpha;
                                m_run = bm;
                                // lower by what the rounding of large offsets
                                // may add, so that p stays below 2^(kLift + kRaise)
                                const float most = fmaf(fabsf(m_run), -0x1p-22f, m_run + (kLift + kRaise));
                                threshold = fmaxf(mx, kBs ? most : most / c);
                                m2 = pair(-m_run, -m_run);
                            }
                            if ((done > 0 || h == 1) && __any_sync(0xffffffffu, raise)) {
                                // the step before's product may still add to O
                                ok = warp_wait(sh, &sh.pv_done[tile], h ^ 1);
                                if (!ok) break;
                                tc::tc_fence_after();
#pragma unroll 1
                                for (int ch = 0; ch < D / 16; ++ch) {
                                    float o[16];
                                    tc::tmem_ld16(col_o + ch * 16, o);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] *= alpha;
                                    tc::tmem_st16(col_o + ch * 16, o);
                                }
                            }
                            if (kBs && __builtin_expect(low_scale(bs), 0))
                                l += low_page_sum(col_s + h * kHalf, left, cb, m_run == -INFINITY ? 0.f : -m_run);
                        }
                        const uint64_t off2 = kBs ? add2(m2, pair(bs.lg_v, bs.lg_v)) : m2;
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float x0, x1;
                                unpair(fma2(pair(x[ch * 32 + 2 * i], x[ch * 32 + 2 * i + 1]), c2, off2), x0, x1);
                                const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
                                sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
                                pk[i] = pack2(p0, p1, kBf16);
                            }
                            tmem_st16u(col_s + h * kHalf + ch * 16, pk);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    warp_arrive(&sh.p_full[tile][h], lane);
                    float l0, l1;
                    unpair(add2(sum[0], sum[1]), l0, l1);
                    l = kBs ? fmaf(l0 + l1, bs.inv_v, l) : l + (l0 + l1);
                }
                ++done;
                ++n_s;
            }
            if (!ok) break;
            // a row without an offset: it read nothing (l = 0, zeros); NaN
            // logits (l is NaN, and stays so with any offset); or keys whose
            // logits are all -inf, which weigh nothing beside other keys but
            // have no softmax of their own: marked by l = 1
            if (m_run == -INFINITY && seen) {
                if (l == 0.f) l = 1.f;
                else m_run = 0.f;
            }

            // ------------------------------------------------- epilogue
            if (own > 0) {
                ok = warp_wait(sh, &sh.o_full[tile], n_o & 1);
                if (!ok) break;
                ++n_o;
                tc::tc_fence_after();
            }
            float w_own = 1.f, w_other = 0.f;  // weights of the two tiles' O in a dual unit
            if (dual) {
                if (tile == 1) {
                    // the first tile joins: the same rows lie in the same lanes
                    sh.dual_stats[r] = make_float2(m_run, l);
                    tc::tc_fence_before();
                    warp_arrive(&sh.dual_ready, lane);
                    warp_arrive(&sh.u_empty[n & 1], lane);
                    continue;
                }
                ok = warp_wait(sh, &sh.dual_ready, n_dual & 1);
                if (!ok) break;
                ++n_dual;
                tc::tc_fence_after();
                const float2 other = sh.dual_stats[r];
                const float m = fmaxf(m_run, other.x);
                if (m != -INFINITY) {
                    float l_other = other.y;  // a NaN stays one, whatever its weight
                    w_own = kBs ? rescale(l, m_run - m) : tc::ex2(m_run - m);
                    w_other = kBs ? rescale(l_other, other.x - m) : tc::ex2(other.x - m);
                    l = kBs ? l + l_other : l * w_own + l_other * w_other;
                    m_run = m;
                } else {
                    l += other.y;
                }
            }
            if (own > 0 && u.marked != 0) {
                take_marked<D, F8>(t, u, tile, have && chosen ? lim : 0, bits, col_o, w_own, w_other);
                w_own = 1.f, w_other = 0.f;
            }
            const bool split = u.pieces > 1;
            const bool none = own == 0 || m_run == -INFINITY;  // no key of this piece was read
            const int64_t prow = static_cast<int64_t>(u.part) * 256 + tile * kRows + r;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (u.tok0 + j_tok) * a.o_s0 +
                                 static_cast<int64_t>(u.h * t.G + g) * a.o_s1;
            const bool vec = a.o_s2 == 1 && (reinterpret_cast<uintptr_t>(out) & 31) == 0;
            const float f = none ? (l > 0.f ? NAN : 0.f) : a.v_scale / l;
            // 32 dims at a time: 64 cost 2 % of a small batch, in instructions to fetch
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                if (own > 0) {
                    tmem_ld32(col_o + c0, o);
                    tc::tmem_wait_ld();
                    if (dual) {
                        float x[32];
                        tmem_ld32(col_o + 128 + c0, x);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(o[i], w_own, x[i] * w_other);
                    }
                    if (c0 + 32 == D) {  // the next unit's products may overwrite O
                        tc::tc_fence_before();
                        warp_arrive(&sh.o_free[tile], lane);
                        if (dual) warp_arrive(&sh.o_free[1], lane);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i];
                } else {
                    // defined on every path: a register that is not would
                    // stay reserved through the block loop
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (have && split) {
                    float *part = reinterpret_cast<float *>(t.ws + t.lay.partials) + prow * D + c0;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store32(part + i, reinterpret_cast<const uint32_t *>(o + i));
                } else if (have && vec) {
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = pack2(o[i + 2 * k] * f, o[i + 2 * k + 1] * f, true);
                        store32(out + c0 + i, w);
                    }
                } else if (have) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) out[(c0 + i) * a.o_s2] = __float2bfloat16_rn(o[i] * f);
                }
            }
            if (have && split) reinterpret_cast<float2 *>(t.ws + t.lay.stats)[prow] = make_float2(m_run, l);
            warp_arrive(&sh.u_empty[n & 1], lane);
        }
    } else {
        tc::regs_dec<kRegsOther>();
        if (warp < kWarpTma) {
            // ------------------------------------------- widen and scrub
            const int row = (warp - kWarpSide) * 32 + lane;  // key of the page; query row of each tile
            Ring<S::kKs> rk;
            Ring<S::kVs> rv;
            Ring<F8 ? S::kRs : 1> rr;
            uint32_t nq = 0;  // units with products
            // this thread's key of the next E4M3 page to f16, into the 16-bit
            // page at `page16`, 64 dims at a time; with `scrub` zeros where no
            // row reads it, and in place of NaN: returns whether there was one
            auto widen = [&](uint8_t *page16, bool scrub, bool unread) {
                const uint8_t *src = smem + S::kOffRaw + rr.slot * S::kPage8 + row * D;
                uint32_t any = 0;
#pragma unroll 1
                for (int b = 0; b < S::kBoxes; ++b) {
                    uint4 w[4];
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
                        w[ch] = *reinterpret_cast<const uint4 *>(
                            src + (((4 * b + ch) ^ (D == 128 ? (row & 7) : ((row >> 1) & 3))) << 4));
                    if (scrub) {
                        uint32_t bad = 0;  // bit 7 of a byte: 127 + 1, a NaN
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
                            const uint32_t *wp = reinterpret_cast<const uint32_t *>(&w[ch]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) bad |= (wp[i] & 0x7f7f7f7fu) + 0x01010101u;
                        }
                        bad &= 0x80808080u;
                        any |= bad;
                        if (unread || bad != 0) {
#pragma unroll
                            for (int ch = 0; ch < 4; ++ch) {
                                uint32_t *wp = reinterpret_cast<uint32_t *>(&w[ch]);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    wp[i] = unread ? 0u : wp[i] & ~__vcmpeq4(wp[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            }
                        }
                    }
                    uint8_t *box = page16 + b * kBox + row * 128;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t h[8];
                        const uint32_t *wp = reinterpret_cast<const uint32_t *>(&w[ch]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) tc::e4m3x4_to_f16x4(wp[i], h[2 * i], h[2 * i + 1]);
                        *reinterpret_cast<uint4 *>(box + (((2 * ch) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(box + (((2 * ch + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                }
                tc::fence_proxy_async();
                warp_arrive(&sh.r_empty[rr.slot], lane);
                rr.next();
                return any != 0 && !unread;
            };
            for (uint32_t n = 0;; ++n) {
                UnitRec &u = sh.unit[n & 1];
                if (!warp_wait(sh, &sh.u_full[n & 1], (n >> 1) & 1) || u.nblk < 0) break;
                const int nblk = u.nblk;
                bool ok = true;
                if (F8 && nblk > 0) {
                    ok = warp_wait(sh, &sh.q_full, nq & 1);
                    if (!ok) break;
                    // a tile that is not there is ready too: its barrier keeps
                    // step with the units
                    for (int tile = 0; tile < 2; ++tile) {
                        float factor = 1.f;
                        if (tile >= u.tiles) factor = 0.f;
                        else if (M == kModeTerms) factor = split_query_row(smem + S::kOffQ + tile * S::kTileQ + row * 128, row);
                        else if (!t.q_f16) factor = halve_query_row<D>(smem + S::kOffQ + tile * S::kTileQ + row * 128, row);
                        sh.row_factor[nq & 1][tile * kRows + row] = factor;
                        tc::fence_proxy_async();
                        warp_arrive(&sh.q_ready[nq & 1][tile], lane);
                    }
                    ++nq;
                }
                for (int j = 0; j < nblk; ++j) {
                    const uint32_t entry = u.kb[j];
                    const int kb = entry & kBlockMask;
                    // V of a page that some row of a tile that takes it does not read in full
                    const bool scrub = (u.mixed & (entry >> kTakeShift)) != 0 || (kb + 1) * kKeys > u.lim_lo;
                    const bool unread = kb * kKeys + row >= u.lim_hi;  // by every row
                    bool mark = false;
                    if (M == kModeWide) {
                        ok = warp_wait(sh, &sh.r_full[rr.slot], rr.parity()) &&
                             (rk.round == 0 || warp_wait(sh, &sh.k_empty[rk.slot], rk.parity() ^ 1));
                        if (!ok) break;
                        widen(smem + S::kOffK + rk.slot * S::kPageK, false, false);
                        warp_arrive(&sh.k_full[rk.slot], lane);
                        rk.next();
                    }
                    if (F8) {
                        ok = warp_wait(sh, &sh.r_full[rr.slot], rr.parity()) &&
                             (rv.round == 0 || warp_wait(sh, &sh.v_empty[rv.slot], rv.parity() ^ 1));
                        if (!ok) break;
                        mark = widen(smem + S::kOffV + rv.slot * S::kPage16, scrub, unread);
                    } else {
                        ok = warp_wait(sh, &sh.v_full[rv.slot], rv.parity());
                        if (!ok) break;
                        uint8_t *dst = smem + S::kOffV + rv.slot * S::kPage16 + row * 128;
                        if (scrub) {
                            uint32_t bad = 0;  // bit 15 of a half: exponent 255 + 1
                            if (!unread) {
#pragma unroll
                                for (int b = 0; b < S::kBoxes; ++b)
#pragma unroll 4
                                    for (int ch = 0; ch < 8; ++ch) {
                                        const uint4 w = *reinterpret_cast<const uint4 *>(dst + b * kBox + ((ch ^ (row & 7)) << 4));
                                        bad |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                                               ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
                                    }
                            }
                            mark = (bad & 0x80008000u) != 0;
                            if (unread || mark) {
#pragma unroll
                                for (int b = 0; b < S::kBoxes; ++b)
#pragma unroll 2
                                    for (int ch = 0; ch < 8; ++ch) {
                                        uint4 *at = reinterpret_cast<uint4 *>(dst + b * kBox + ((ch ^ (row & 7)) << 4));
                                        uint4 w = unread ? make_uint4(0, 0, 0, 0) : *at;
                                        uint32_t *wp = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            if (!finite_bits(wp[i], true)) wp[i] &= 0xffff0000u;
                                            if (!finite_bits(wp[i] >> 16, true)) wp[i] &= 0xffffu;
                                        }
                                        *at = w;
                                    }
                            }
                            tc::fence_proxy_async();
                        }
                    }
                    if (mark) {
                        atomicOr(&u.marks[kb >> 5], 1u << (kb & 31));
                        *reinterpret_cast<volatile int32_t *>(&u.marked) = 1;
                    }
                    warp_arrive(&sh.v_ready[rv.slot], lane);
                    rv.next();
                }
                if (!ok) break;
                warp_arrive(&sh.u_empty[n & 1], lane);
            }
        } else if (warp == kWarpTma) {
            // ------------------------------------------------- TMA loads
            if (lane == 0) {
                Ring<S::kKs> rk;
                Ring<S::kVs> rv;
                Ring<F8 ? S::kRs : 1> rr;
                uint32_t nq = 0, n_pages = 0;
                bool ok = true;
                // the next page of a ring, once its slot's last round has been read
                auto room = [&](const auto &ring, uint64_t *empty) {
                    return !aborted(sh) && (ring.round == 0 || wait_or_abort(sh, &empty[ring.slot], ring.parity() ^ 1));
                };
                auto copy8 = [&](const CUtensorMap *map, uint8_t *dst, uint64_t *full, int h, int slot0) {
                    tc::mbar_arrive_expect_tx(full, S::kPage8);
                    tc::tma_load_3d(dst, map, full, 0, h, slot0);
                };
                auto copy16 = [&](const CUtensorMap *map, uint8_t *dst, uint64_t *full, int h, int slot0) {
                    tc::mbar_arrive_expect_tx(full, S::kPage16);
                    for (int b = 0; b < S::kBoxes; ++b) tc::tma_load_3d(dst + b * kBox, map, full, 64 * b, h, slot0);
                };
                for (uint32_t n = 0; ok; ++n) {
                    UnitRec &u = sh.unit[n & 1];
                    ok = wait_or_abort(sh, &sh.u_full[n & 1], (n >> 1) & 1);
                    if (!ok || u.nblk < 0) break;
                    const int nblk = u.nblk;
                    for (int j = 0; j < nblk && ok; ++j) {
                        const int slot0 = u.page[j] * kKeys;
                        if (M == kModeWide) {
                            ok = room(rr, sh.r_empty);
                            if (!ok) break;
                            copy8(&tmap_k, smem + S::kOffRaw + rr.slot * S::kPage8, &sh.r_full[rr.slot], u.h, slot0);
                            if (kBs) load_block_scale(&sh.scale[n_pages++ % kScaleRing], a.sc, u.page[j], u.h, &sh.r_full[rr.slot]);
                            rr.next();
                        } else {
                            ok = room(rk, sh.k_empty);
                            if (!ok) break;
                            uint8_t *dst = smem + S::kOffK + rk.slot * S::kPageK;
                            if (M == kModeTerms) copy8(&tmap_k, dst, &sh.k_full[rk.slot], u.h, slot0);
                            else copy16(&tmap_k, dst, &sh.k_full[rk.slot], u.h, slot0);
                            if (kBs) load_block_scale(&sh.scale[n_pages++ % kScaleRing], a.sc, u.page[j], u.h, &sh.k_full[rk.slot]);
                            rk.next();
                        }
                        if (j == 0) {
                            // the queries, once the last unit's products have read theirs
                            ok = nq == 0 || wait_or_abort(sh, &sh.q_empty, (nq - 1) & 1);
                            if (!ok) break;
                            const int tiles = u.tiles;
                            tc::mbar_arrive_expect_tx(&sh.q_full, tiles * S::kBoxes * 128 * t.G * t.lay.tt);
                            for (int i = 0; i < tiles; ++i)
                                for (int b = 0; b < S::kBoxes; ++b)
                                    tc::tma_load_3d(smem + S::kOffQ + i * S::kTileQ + b * kBox, &tmap_q, &sh.q_full, 64 * b,
                                                    u.h * t.G, u.tok0 + (u.dual ? 0 : i * t.lay.tt));
                            ++nq;
                        }
                        if (F8) {
                            ok = room(rr, sh.r_empty);
                            if (!ok) break;
                            copy8(&tmap_v, smem + S::kOffRaw + rr.slot * S::kPage8, &sh.r_full[rr.slot], u.h, slot0);
                            if (M == kModeWide && kBs) tc::mbar_arrive(&sh.r_full[rr.slot]);  // no scales beside V
                            rr.next();
                        } else {
                            ok = room(rv, sh.v_empty);
                            if (!ok) break;
                            copy16(&tmap_v, smem + S::kOffV + rv.slot * S::kPage16, &sh.v_full[rv.slot], u.h, slot0);
                            rv.next();
                        }
                    }
                    if (ok) tc::mbar_arrive(&sh.u_empty[n & 1]);
                }
                // every issued copy lands before the CTA may exit; only after
                // an abort can one still be in flight
                if (!ok) {
                    if (nq > 0) tc::mbar_wait_tries(&sh.q_full, (nq - 1) & 1);
                    auto landed = [&](const auto &ring, uint64_t *full, int slots) {
                        for (int i = 0; i < slots; ++i) {
                            // the last round of slot i that was begun
                            const uint32_t rounds = ring.round + (static_cast<uint32_t>(i) < ring.slot ? 1 : 0);
                            if (rounds > 0) tc::mbar_wait_tries(&full[i], (rounds - 1) & 1);
                        }
                    };
                    if (M != kModeWide) landed(rk, sh.k_full, S::kKs);
                    if (F8) landed(rr, sh.r_full, S::kRs);
                    else landed(rv, sh.v_full, S::kVs);
                }
            }
        } else if (warp == kWarpMma || warp == kWarpMma1) {
            // ----------------------------------------------- MMA issuers
            // One warp per tile: a product takes 256 to 384 tensor cycles and
            // the pipe's queue holds few instructions, so what a warp does
            // between two products (waits, commits: 100 to 300 cycles) would
            // leave the pipe idle if the other tile's products did not fill
            // it.  The whole warp waits and counts, one elected lane issues.
            const int i = warp == kWarpMma ? 0 : 1;
            const uint32_t idesc_s = M == kModeTerms ? tc::idesc_m128(kHalf, false, false) : tc::idesc_f16_m128(kHalf, kBf16);
            const uint32_t idesc_o = tc::idesc_f16_m128(D, kBf16) | (1u << 16);  // B (V) MN-major
            const uint32_t q_low = desc_low(tc::smem_u32(smem + S::kOffQ + i * S::kTileQ), 16);
            const uint32_t k_low = desc_low(tc::smem_u32(smem + S::kOffK), 16);
            const uint32_t v_low = desc_low(tc::smem_u32(smem + S::kOffV), kBox);
            const uint32_t col_s = tmem + kColS + i * 128, col_o = tmem + kColO + i * 128;
            Ring<S::kKs> rk;
            Ring<S::kVs> rv;
            uint32_t nq = 0, n_p = 0, n_o = 0;  // units with products, P and O tiles so far
            bool ok = true;
            auto wait_k = [&] { return warp_wait(sh, &sh.k_full[rk.slot], rk.parity()); };
            auto wait_v = [&] { return warp_wait(sh, &sh.v_ready[rv.slot], rv.parity()); };
            auto wait_q = [&] {
                return F8 ? warp_wait(sh, &sh.q_ready[nq & 1][i], (nq >> 1) & 1) : warp_wait(sh, &sh.q_full, nq & 1);
            };
            // S = Q K^T over one half of the page's keys; `last`: the unit's last use of the queries
            auto qk = [&](int half, bool last) {
                const uint32_t k = k_low + rk.slot * (S::kPageK >> 4) + half * (kHalf * 128 >> 4);
                tc::tc_fence_after();
                if (elect_one()) {
                    if (M == kModeTerms) {
                        // 32 dims a step: 32 bytes into K's row, 64 into the queries', the second terms 32 on
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ss<true>(col_s + half * kHalf,
                                         q_low + (ks >> 2) * (kBox >> 4) + ((ks >> 1) & 1) * (64 >> 4) + (ks & 1) * (32 >> 4),
                                         k + (ks >> 1) * (32 >> 4), idesc_s, ks > 0);
                    } else {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            // 16 dims a step: 32 bytes into a 128-byte row, the next 64 dims one box on
                            const uint32_t off = ((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                            mma_ss<false>(col_s + half * kHalf, q_low + off, k + off, idesc_s, ks > 0);
                        }
                    }
                    tc::mma_commit(&sh.s_full[i][half]);
                    if (half == 1) tc::mma_commit(&sh.k_empty[rk.slot]);
                    if (last) tc::mma_commit(&sh.q_empty);
                }
                __syncwarp();
                if (half == 1) rk.next();
            };
            // O (+)= P V over one half of the page's keys; `last`: O is complete
            auto pv = [&](int half, bool add, bool last) {
                const uint32_t v = v_low + rv.slot * (S::kPage16 >> 4) + half * (kHalf * 128 >> 4);
                tc::tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kHalf / 16; ++ks)
                        // P: 16 keys = 8 columns of 16-bit pairs; V: two 8-key groups, the next 64 dims one box on
                        mma_ts(col_o, col_s + half * kHalf + ks * 8, v + ks * (2048 >> 4), idesc_o, ks > 0 || add);
                    tc::mma_commit(&sh.pv_done[i]);
                    if (last) tc::mma_commit(&sh.o_full[i]);
                    if (half == 1) tc::mma_commit(&sh.v_empty[rv.slot]);
                }
                __syncwarp();
                if (half == 1) rv.next();
            };
            for (uint32_t n = 0; ok; ++n) {
                UnitRec &u = sh.unit[n & 1];
                ok = warp_wait(sh, &sh.u_full[n & 1], (n >> 1) & 1);
                if (!ok || u.nblk < 0) break;
                const int nblk = u.nblk;
                const int own = i < u.tiles ? u.own[i] : 0;
                const bool dual = u.dual != 0;
                // pages that this tile does not take only pass by
                int k_at = 0, v_at = 0;  // next K and V page in the rings
                auto pass_k = [&](int to) {
                    for (; k_at < to && ok; ++k_at) {
                        ok = wait_k();
                        if (ok && lane == 0) tc::mbar_arrive(&sh.k_empty[rk.slot]);
                        rk.next();
                    }
                };
                auto pass_v = [&](int to) {
                    for (; v_at < to && ok; ++v_at) {
                        ok = wait_v();
                        if (ok && lane == 0) tc::mbar_arrive(&sh.v_empty[rv.slot]);
                        rv.next();
                    }
                };
                auto next_own = [&](int j) {
                    while (!((u.kb[j] >> (kTakeShift + i)) & 1u)) ++j;
                    return j;
                };
                // Pages come in the order K, V, K, V, and a ring holds few: where
                // more than one passes by, both of each have to, in that order,
                // or the copies would wait for this warp and it for them.
                auto pass = [&](int to) {
                    while (ok && (k_at < to || v_at < to)) {
                        if (k_at <= v_at) pass_k(k_at + 1);
                        else pass_v(v_at + 1);
                    }
                };
                if (own > 0 && own == nblk) {
                    // every page, the common case: nothing but the products
                    // between one wait and the next
                    ok = wait_q() && wait_k();
                    if (!ok) break;
                    qk(0, false);
                    qk(1, nblk == 1);
                    for (int j = 0; j < nblk && ok; ++j) {
                        const bool last = j == nblk - 1;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h == 0) ok = wait_v() && (j > 0 || n_o == 0 || warp_wait(sh, &sh.o_free[i], (n_o - 1) & 1));
                            ok = ok && warp_wait(sh, &sh.p_full[i][h], n_p & 1);
                            if (!ok) break;
                            pv(h, j > 0 || h > 0, h == 1 && last);
                            if (last) continue;
                            // the next page's half into the buffer that this half's P leaves
                            if (h == 0) ok = wait_k();
                            if (!ok) break;
                            qk(h, h == 1 && j == nblk - 2);
                        }
                        ++n_p;
                    }
                    ++n_o;
                    k_at = v_at = nblk;
                } else if (own > 0) {
                    int j = dual ? i : next_own(0);
                    if (j > 1) pass(j);
                    else pass_k(j);
                    ok = ok && wait_q() && wait_k();
                    if (!ok) break;
                    qk(0, false);
                    qk(1, own == 1);
                    ++k_at;
                    for (int done = 0; done < own && ok; ++done) {
                        const bool last = done == own - 1;
                        const int next = last ? nblk : (dual ? j + 2 : next_own(j + 1));
                        const bool near = !last && next - j <= 2;
                        pass_v(j);
                        ok = ok && wait_v() && (done > 0 || n_o == 0 || warp_wait(sh, &sh.o_free[i], (n_o - 1) & 1)) &&
                             warp_wait(sh, &sh.p_full[i][0], n_p & 1);
                        if (!ok) break;
                        pv(0, done > 0, false);
                        if (near) {
                            // the next page's half into the buffer that this half's P leaves
                            pass_k(next);
                            ok = ok && wait_k();
                            if (!ok) break;
                            qk(0, false);
                        }
                        ok = warp_wait(sh, &sh.p_full[i][1], n_p & 1);
                        if (!ok) break;
                        pv(1, true, last);
                        ++v_at;
                        ++n_p;
                        if (last) {
                            ++n_o;
                            break;
                        }
                        if (!near) {
                            pass(next);
                            ok = ok && wait_k();
                            if (!ok) break;
                            qk(0, false);
                        }
                        qk(1, done == own - 2);
                        ++k_at;
                        j = next;
                    }
                } else if (nblk > 0) {
                    // nothing to multiply: the queries, too, only pass by, but
                    // not before their terms are written in place: the next
                    // unit's queries are copied over them behind this arrival,
                    // and a unit of one page that the other tile takes has
                    // nothing else that waits for this tile's
                    ok = wait_q();
                    if (ok && lane == 0) tc::mbar_arrive(&sh.q_empty);
                }
                if (ok) pass(nblk);
                if (!ok) break;
                if (nblk > 0) ++nq;
                warp_arrive(&sh.u_empty[n & 1], lane);
            }
            // every issued product completes before tensor memory is released
            if (elect_one()) tc::mma_commit(&sh.drain[i]);
            __syncwarp();
            tc::mbar_wait_tries(&sh.drain[i], 0);
        } else if (warp == kWarpSched) {
            // ---------------------------------------------- units, page lists
            const ChunkPair *pairs = reinterpret_cast<const ChunkPair *>(t.ws + t.lay.pairs);
            const int32_t n_units = hd->n_units, n_pairs = hd->n_pairs, head_parts = hd->head_parts;
            // the pair whose units of one head hold v, and its key, by 32-way search
            auto pair_of = [&](int32_t v, ChunkKey &key) {
                int lo = 0, span = n_pairs;
                do {
                    const int step = (span + 31) / 32, at = lo + lane * step;
                    int4 k = make_int4(0, 0, 0, 0);
                    if (lane * step < span) k = *reinterpret_cast<const int4 *>(&pairs[at].key);
                    const bool below = lane * step < span && k.x <= v;
                    const int last = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);  // lane 0 is below
                    key.unit0 = __shfl_sync(0xffffffffu, k.x, last);
                    key.seq0 = __shfl_sync(0xffffffffu, k.y, last);
                    key.seq_units = __shfl_sync(0xffffffffu, k.z, last);
                    key.pieces = __shfl_sync(0xffffffffu, k.w, last);
                    lo += last * step;
                    span = min(step, span - last * step);
                } while (span > 1);
                return lo;
            };
            int32_t id = blockIdx.x;
            for (uint32_t n = 0;; ++n) {
                UnitRec &u = sh.unit[n & 1];
                if (n >= 2 && !warp_wait(sh, &sh.u_empty[n & 1], ((n >> 1) - 1) & 1)) break;
                if (aborted(sh)) break;
                if (id >= n_units) {
                    if (lane == 0) {
                        u.nblk = -1;
                        tc::mbar_arrive(&sh.u_full[n & 1]);
                    }
                    break;
                }
                // sequence, then head, then the unit among the sequence's
                // (each load that waits for another costs the first unit 0.4 us:
                // a search brings the key along, a pair record all of its sequence)
                ChunkKey key;
                pair_of(id / a.Hkv, key);
                const int32_t rest = id - key.seq0 * a.Hkv;
                const int h = rest / key.seq_units, v = key.seq0 + rest % key.seq_units;
                const ChunkPair pr = pairs[pair_of(v, key)];
                const int piece = v - key.unit0, pieces = key.pieces;
                const int32_t table_row = pr.row, pre = pr.pre, cap = pr.cap;
                const int32_t lim_lo = max(min(pre + pr.i0 + 1, cap), 0);
                const int32_t lim_hi = max(min(pre + pr.i0 + pr.nt, cap), 0);
                const int vis = (lim_hi + kKeys - 1) / kKeys;  // blocks that the last token sees
                // blocks of the pair: all that it sees, or the union of its query blocks' selections
                // lane l holds blocks 32 l ..
                auto below = [&](int blocks) -> uint32_t {
                    return lane * 32 >= blocks ? 0u : (blocks - lane * 32 >= 32 ? 0xffffffffu : (1u << (blocks - lane * 32)) - 1u);
                };
                const int nt0 = min(pr.nt, t.lay.tt);  // tokens of the first tile
                uint32_t words[2] = {below(vis), pr.nt > nt0 ? below(vis) : 0u};
                int32_t qrow0 = 0, qrow_end = 0, mixed = 0;
                if (a.tk != nullptr) {
                    qrow0 = a.cub[pr.b * a.cub_s0];
                    qrow_end = min(a.cub[(pr.b + 1) * a.cub_s0], a.n_rows);
                    for (int i = 0; i < 2; ++i) {
                        // the union of the selections of the tile's query blocks
                        const int from = i == 0 ? 0 : nt0, to = i == 0 ? nt0 : pr.nt;
                        if (from >= to) continue;
                        const int q0 = (pr.i0 + from) / a.bsq, q1 = (pr.i0 + to - 1) / a.bsq;
                        uint32_t any = 0;
                        if (lane < t.lay.words) {
                            const uint32_t *bm = reinterpret_cast<const uint32_t *>(t.ws + t.lay.bitmaps) +
                                                 (t.heads_built > 1 ? static_cast<int64_t>(h) : 0) * a.n_rows * t.lay.words + lane;
#pragma unroll 4
                            for (int q = q0; q <= q1; ++q) {
                                const int64_t row = static_cast<int64_t>(qrow0) + q;
                                if (row >= 0 && row < qrow_end) any |= bm[row * t.lay.words];
                            }
                        }
                        words[i] &= any;
                        if (q1 > q0) mixed |= 1 << i;
                    }
                }
                const uint32_t word = words[0] | words[1];
                // this piece's share of the list, by rank
                int before = __popc(word);
                const int mine = before;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, before, d);
                    if (lane >= d) before += y;
                }
                const int listed = __shfl_sync(0xffffffffu, before, 31);
                before -= mine;
                const int r0 = static_cast<int>(static_cast<int64_t>(listed) * piece / pieces);
                const int r1 = static_cast<int>(static_cast<int64_t>(listed) * (piece + 1) / pieces);
                int count = 0, own0 = 0, own1 = 0;
                for (int w = 0; w * 32 < vis; ++w) {
                    const uint32_t ww = __shfl_sync(0xffffffffu, word, w);
                    const uint32_t w0 = __shfl_sync(0xffffffffu, words[0], w), w1 = __shfl_sync(0xffffffffu, words[1], w);
                    const int wb = __shfl_sync(0xffffffffu, before, w);
                    if (wb >= r1 || wb + __popc(ww) <= r0) continue;
                    const int rank = wb + __popc(ww & ((1u << lane) - 1u));
                    bool take = ((ww >> lane) & 1u) && rank >= r0 && rank < r1;
                    int32_t page = -1;
                    if (take) page = a.bt[table_row * a.bt_s0 + (w * 32 + lane) * a.bt_s1];
                    take = take && page >= 0 && page < a.P;
                    const uint32_t taken = __ballot_sync(0xffffffffu, take);
                    if (take) {
                        const int at = count + __popc(taken & ((1u << lane) - 1u));
                        u.page[at] = page;
                        const uint32_t tiles = ((w0 >> lane) & 1u) | (((w1 >> lane) & 1u) << 1);
                        u.kb[at] = static_cast<uint16_t>((w * 32 + lane) | (tiles << kTakeShift));
                    }
                    count += __popc(taken);
                    own0 += __popc(taken & w0);
                    own1 += __popc(taken & w1);
                }
                const bool dual = pr.nt <= t.lay.tt && count >= 2;
                if (dual) {
                    __syncwarp();
                    for (int at = lane; at < count; at += 32)
                        u.kb[at] = static_cast<uint16_t>((u.kb[at] & kBlockMask) | ((1u + (at & 1)) << kTakeShift));
                    own0 = (count + 1) / 2;
                    own1 = count / 2;
                    mixed = mixed ? 3 : 0;
                }
                u.marks[lane] = 0;
                if (lane == 0) {
                    u.nblk = count;
                    u.tok0 = pr.tok0;
                    u.i0 = pr.i0;
                    u.nt = pr.nt;
                    u.h = h;
                    u.dual = dual;
                    u.tiles = dual || pr.nt > t.lay.tt ? 2 : 1;
                    u.own[0] = own0;
                    u.own[1] = own1;
                    u.pre = pre;
                    u.cap = cap;
                    u.lim_lo = lim_lo;
                    u.lim_hi = lim_hi;
                    u.mixed = mixed;
                    u.qrow0 = qrow0;
                    u.qrow_end = qrow_end;
                    u.pieces = pieces;
                    u.part = h * head_parts + pr.part0 + piece;
                    u.marked = 0;
                }
                warp_arrive(&sh.u_full[n & 1], lane);
                if (lane == 0) id = static_cast<int32_t>(gridDim.x) + atomicAdd(&hd->next_unit, 1);
                id = __shfl_sync(0xffffffffu, id, 0);
            }
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (threadIdx.x == 0 && aborted(sh)) atomicOr(&hd->status, 1);
    if (warp == kWarpMma) tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the pieces of split pairs, in piece order: a warp takes kJoinRows
// neighbouring rows of one head at a time.  A share of the lanes finds each
// row's offset and sum from the pieces' statistics; then the rows' partials, a
// lane per D / 32 dims, are added with no load waiting for another, so a group
// costs a few memory latencies however many pieces it has.  (Joined by the last
// piece's softmax warps, thread by thread, the rows of 10 pieces took 150 us.)
constexpr int kJoinRows = 2;
constexpr int kJoinLanes = 32 / kJoinRows;

template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ TcArgs t) {
    tc::pdl_wait();
    const ChunkArgs &a = t.a;
    const ChunkHeader *hd = reinterpret_cast<const ChunkHeader *>(t.ws + t.lay.header);
    const int4 *splits = reinterpret_cast<const int4 *>(t.ws + t.lay.splits);  // of ChunkSplit
    const int lane = threadIdx.x & 31;
    constexpr int kGroups = 256 / kJoinRows;  // of a pair and head
    // the first record is on its way with the header, whether there is one or not
    // (at most kChunkMaxParts / 2 pairs and heads are split)
    uint32_t k = blockIdx.x * 8 + (threadIdx.x >> 5);
    auto record = [&](uint32_t at) {
        const uint32_t i = at / kGroups / a.Hkv;
        return i < t.lay.pair_cap ? splits[i] : make_int4(0, 0, 0, 0);
    };
    int4 next = record(k);
    const uint32_t groups = hd->n_splits * a.Hkv * kGroups, stride = gridDim.x * 8;
    constexpr int kPer = D / 32;
    for (; k < groups; k += stride) {
        const int r0 = static_cast<int>(k % kGroups) * kJoinRows;
        const int h = static_cast<int>((k / kGroups) % a.Hkv);
        const ChunkSplit pr = {next.x, next.y, next.z, next.w};
        next = record(k + stride);
        auto token = [&](int r) {  // of the pair, or -1 where the row holds none
            const int j = (r >> 7) * t.lay.tt + (r & 127) / t.G;
            return (r & 127) < t.lay.tt * t.G && j < pr.nt ? j : -1;
        };
        if (token(r0) < 0) continue;  // rows fill a tile from its first on
        const int64_t row0 = (static_cast<int64_t>(h) * hd->head_parts + pr.part0) * 256 + r0;
        const float2 *stats = reinterpret_cast<const float2 *>(t.ws + t.lay.stats) + row0;
        const float *parts = reinterpret_cast<const float *>(t.ws + t.lay.partials) + row0 * D + lane * kPer;
        // offset and sum of the lane's row
        const int own = lane / kJoinLanes;
        const bool mine = token(r0 + own) >= 0;
        float M = -INFINITY, L = 0.f;
        for (int p = lane % kJoinLanes; p < pr.pieces; p += kJoinLanes)
            if (mine) M = fmaxf(M, stats[p * 256 + own].x);
#pragma unroll
        for (int d = kJoinLanes / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        for (int p = lane % kJoinLanes; p < pr.pieces; p += kJoinLanes)
            if (mine) {
                const float2 s = stats[p * 256 + own];
                // a NaN stays one, whatever its weight
                float y = s.y;
                if (M != -INFINITY) {
                    if (a.sc.k != nullptr) rescale(y, s.x - M);
                    else y *= tc::ex2(s.x - M);
                }
                L += y;
            }
#pragma unroll
        for (int d = kJoinLanes / 2; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            const int j = token(r0 + i);
            const float m = __shfl_sync(0xffffffffu, M, kJoinLanes * i), l = __shfl_sync(0xffffffffu, L, kJoinLanes * i);
            if (j < 0) continue;
            float o[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] = 0.f;
#pragma unroll 4
            for (int p = 0; p < pr.pieces; ++p) {
                const float w = m == -INFINITY ? 0.f : tc::ex2(stats[p * 256 + i].x - m);
                const float *src = parts + (static_cast<int64_t>(p) * 256 + i) * D;
                float x[kPer];
                if (kPer == 4) *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(src);
                else *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(src);
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = fmaf(x[e], w, o[e]);
            }
            // without an offset: nothing read, or logits that are all -inf
            const float f = m == -INFINITY ? (l > 0.f ? NAN : 0.f) : a.v_scale / l;
            const int g = ((r0 + i) & 127) % t.G;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + static_cast<int64_t>(pr.tok0 + j) * a.o_s0 +
                                 static_cast<int64_t>(h * t.G + g) * a.o_s1;
            if (a.o_s2 == 1 && (reinterpret_cast<uintptr_t>(out) & 7) == 0) {
                uint32_t w[kPer / 2];
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) w[e] = pack2(o[2 * e] * f, o[2 * e + 1] * f, true);
                if (kPer == 4) reinterpret_cast<uint2 *>(out)[lane] = make_uint2(w[0], w[kPer / 2 - 1]);
                else reinterpret_cast<uint32_t *>(out)[lane] = w[0];
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) out[(lane * kPer + e) * a.o_s2] = __float2bfloat16_rn(o[e] * f);
            }
        }
    }
}

// [rows, heads, D] tensor as a 3-D map: boxes of `dims` dims x `heads_box`
// heads x `rows_box` rows, swizzled over the box's row width.
bool make_map(CUtensorMap *m, CUtensorMapDataType type, int es, const void *base, int64_t D, int64_t heads, int64_t rows,
              int64_t s1, int64_t s0, int dims, int heads_box, int rows_box) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t shape[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * es, static_cast<cuuint64_t>(s0) * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(dims), static_cast<cuuint32_t>(heads_box),
                               static_cast<cuuint32_t>(rows_box)};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(m, type, 3, const_cast<void *>(base), shape, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              dims * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Strides of extents above one must be positive multiples of 16 bytes below
// the map's limit of 2^40 bytes.
bool map_ok(const void *base, int es, int64_t s0, int64_t s1, int64_t n0, int64_t n1) {
    auto legal = [es](int64_t s) { return s > 0 && (s * es) % 16 == 0 && s < (int64_t(1) << 40) / es; };
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (n1 <= 1 || legal(s1)) && (n0 <= 1 || legal(s0));
}

template <int D, Mode M, bool kBs = false>
cudaError_t launch(const ChunkArgs &a, void *ws, cudaStream_t stream, bool *used) {
    using S = Shape<D, M>;
    constexpr bool F8 = S::kF8;
    constexpr int kSmem = S::kEnd + 1024 + static_cast<int>(sizeof(Shared));
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    const int G = a.Hq / a.Hkv;
    const ChunkLayout lay(a.total_q, a.Hq, a.Hkv, a.D, a.B, a.NB, a.n_rows);
    constexpr int es = F8 ? 1 : 2;
    constexpr CUtensorMapDataType kv_type = F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const int64_t slots = a.P * kKeys;
    // strides of extents of one are never stepped over: any legal value does
    const int64_t qs1 = a.Hq > 1 ? a.q_s1 : D, qs0 = a.total_q > 1 ? a.q_s0 : D;
    const int64_t ks1 = a.Hkv > 1 ? a.k_s1 : D, vs1 = a.Hkv > 1 ? a.v_s1 : D;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.q, D, a.Hq, a.total_q, qs1, qs0, 64, G, lay.tt) ||
        !make_map(&mk, kv_type, es, a.k, D, a.Hkv, slots, ks1, a.k_s0, F8 ? D : 64, 1, kKeys) ||
        !make_map(&mv, kv_type, es, a.v, D, a.Hkv, slots, vs1, a.v_s0, F8 ? D : 64, 1, kKeys))
        return cudaSuccess;
    const void *func = reinterpret_cast<const void *>(chunk_tc_kernel<D, M, kBs>);
    cudaError_t e = opt_in_smem(func, kSmem);
    if (e != cudaSuccess) return e;

    ChunkPlanArgs p{};
    p.a = a;
    p.lay = lay;
    p.ws = static_cast<char *>(ws);
    p.heads_built = (a.tk_s0 == 0 || a.Hkv == 1) ? 1 : a.Hkv;
    p.ctas = device_sm_count();
    e = launch_chunk_plan(p, stream);
    if (e != cudaSuccess) return e;

    TcArgs t{};
    t.a = a;
    t.lay = lay;
    t.ws = p.ws;
    t.G = G;
    t.heads_built = p.heads_built;
    t.q_f16 = a.q_dt == SPD_F16;
    t.c = a.sm_scale * a.k_scale * kLog2e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    // the prologue may run beside the plan kernel's tail; the kernel waits for
    // its end before it reads global memory
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, chunk_tc_kernel<D, M, kBs>, mq, mk, mv, t);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(8 * p.ctas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, t);
    if (e != cudaSuccess) return e;
    count_launches(3);
    *used = true;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkArgs &a, void *ws, cudaStream_t stream, bool *used) {
    *used = false;
    const bool f8 = a.kv_dt == SPD_E4M3;
    if (a.D != 64 && a.D != 128) return cudaSuccess;
    if (a.q_dt != SPD_BF16 && !(f8 && a.q_dt == SPD_F16)) return cudaSuccess;
    // the exponents need one sign, and the queries' scaling some headroom
    const float c = a.sm_scale * a.k_scale * kLog2e;
    const bool block = a.sc.k != nullptr;  // whose scales go down to 2^-64 and up to 2^64
    if (!(c > (block ? 1e-10f : 1e-30f)) || !(c < (block ? 1e10f : 1e30f))) return cudaSuccess;
    const int es = f8 ? 1 : 2;
    if (a.P < 1 || a.q_s2 != 1 || !map_ok(a.q, 2, a.q_s0, a.q_s1, a.total_q, a.Hq) ||
        !map_ok(a.k, es, a.k_s0, a.k_s1, a.P * kKeys, a.Hkv) || !map_ok(a.v, es, a.v_s0, a.v_s1, a.P * kKeys, a.Hkv))
        return cudaSuccess;
    if (!f8) return a.D == 128 ? launch<128, kModeBf16>(a, ws, stream, used) : launch<64, kModeBf16>(a, ws, stream, used);
    if (block) {
        if (a.D == 128 && a.q_dt == SPD_BF16) return launch<128, kModeTerms, true>(a, ws, stream, used);
        return a.D == 128 ? launch<128, kModeWide, true>(a, ws, stream, used) : launch<64, kModeWide, true>(a, ws, stream, used);
    }
    // 64-dim terms would need rows of 64 bytes, f16 queries a third term: those are multiplied as f16
    if (a.D == 128 && a.q_dt == SPD_BF16) return launch<128, kModeTerms>(a, ws, stream, used);
    return a.D == 128 ? launch<128, kModeWide>(a, ws, stream, used) : launch<64, kModeWide>(a, ws, stream, used);
}

}  // namespace spd
