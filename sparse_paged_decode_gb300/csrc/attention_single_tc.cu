// attention_single_tc.cu -- paged sparse / dense GQA decode attention of single
// query tokens over block-scaled E4M3 caches, on the sm_103a tensor cores.
//
// For the decode step proper: every query row by itself, G = Hq / Hkv <= 16
// query heads to a kv head.  HBM bounds it, so the kernel is built around the
// loads and everything else is kept below them:
//
//  * Work.  Row t has n_t = ceil(L_t / 128) blocks (at most K of them with a
//    selection, at least one place).  All rows' blocks in one line are cut into
//    equal pieces, one for each team of CTAs; the CTAs of a team take the same
//    blocks, two kv heads each, so a page's slots are read in full at about the
//    same time.  A piece that ends inside a row leaves fp32 partials, which the
//    last piece of the row joins (an atomic ticket, no waiting).  One CTA
//    writes the line's offsets before; a warp of each CTA makes its own block
//    lists, one row ahead.
//
//  * Contractions, keys and dims on the 128 tensor-memory lanes, query heads on
//    columns:
//        S[key][r]  = K[key][:] . q[r][:]     kind::f8f6f4, K as read, q as two
//                     E4M3 terms (bf16; exact within 2^9 of the row's largest
//                     element) or three (f16), side by side along N
//        O[d][r]   += V[:][d] . P[:][r]       kind::f8f6f4, V as read (MN-major),
//                     P as three E4M3 terms side by side
//    With p in [0, 2^8], p = t0 + 2^-5 t1 + 2^-10 t2 where t1 and t2 are the
//    E4M3 roundings of what is left, times 2^5: every rounding is off by 2^-4 of
//    itself or by half of E4M3's smallest step, so p is off by at most 2^-12 of
//    itself, or 2^-20.  The terms' products stay apart (columns of their own) and
//    are added in fp32 at the end.  So V needs no widening to f16, which took the
//    kernels for wider groups four warps and four fifths of their shared-memory
//    traffic.
//
//  * Softmax.  The two heads of a page have a warpgroup each.  A thread holds
//    one key's logits of the kN query heads; offsets (m, in log2 units, with the
//    page's V scale: block_scale.cuh) are raised when a logit runs more than 2^8
//    above, to 2^2 below the block's maximum.
//
// Measured (64 / 8 heads, graph of calls): 16 rows over 16384 keys 86.9 us, 6.2 TB/s
// or 0.91 of the measured copy rate, where the keys-on-lanes kernel (one head a
// unit, V widened, two planner kernels) took 137; 16 rows over 16 selected blocks
// each 22.7 us (34.5); one row over 2048 keys 12.8 us (22.2).  Rows that share
// their blocks read them once each here: 452 rows of 64 requests over 64 of up to
// 128 blocks take 460 us, the query-rows kernel 264.
//
// Roles (12 warps): warp 0 TMA loads, warp 1 issues Q K^T, warp 2 P V, warp 3
// makes the block lists, warps 4-7 and 8-11 the softmax and epilogue of the two
// heads.  Every wait is bounded: one that gives up sets bit 0 of the workspace
// status word and the CTA winds down.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "block_scale.cuh"
#include "plan.cuh"
#include "spd_internal.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace spd {

cudaError_t launch_attention_single(const AttnArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream, bool *used);

namespace {

constexpr int kD = 128;
constexpr int kKeys = kBlock;
constexpr int kThreads = 384;
constexpr int kWarpTma = 0, kWarpQk = 1, kWarpPv = 2, kWarpSoft = 4;  // warp 3: block lists
constexpr int kGroup = 128;        // threads of one head's softmax
constexpr int kStages = 3;
constexpr int kTile = kKeys * kD;  // one head's K or V page, bytes
constexpr int kStage = 4 * kTile;  // K and V of two heads
constexpr int kListCap = 256;      // blocks of a unit (a row's piece may take several)
// A stage is given back once both heads' P V of its page are done: the loader is
// at most three pages ahead of one whose softmax runs.
constexpr int kScaleRing = 4;
constexpr float kCap = 8.f;        // log2 of the largest p
constexpr float kTarget = 2.f;     // where a raise puts the block's maximum
constexpr int kTermShift = 5;      // log2 of a term's scale over the one before
constexpr int kPTerms = 3;
constexpr int kStride = kD + kPartialStride;  // floats of a partial row
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;               // S of head h, buffer k at (2 h + k) * 64; O of head h at kColO + 64 h
constexpr uint32_t kUnitReleases = 3 + 8;     // loader, two issuers, softmax warps

struct Unit {
    int32_t count;       // blocks; -1: no more units
    int32_t row, limit;  // query row and its keys
    int32_t first, last; // of the row's piece
    int32_t part;        // partial slot of this CTA, -1 where the row is whole here
    int32_t team0, n_split, slot0;  // pieces of the row: first team, how many, the first one's slot
    int32_t page[kListCap];
    uint16_t block[kListCap];
};

struct Shared {
    uint64_t u_full[2], u_empty[2];
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t q_full;
    uint64_t s_full[2][2], s_empty[2][2];  // [head][buffer]
    uint64_t p_full[2], pv_done[2];        // [head]
    uint64_t drain[2];
    float2 scale[2][kScaleRing];
    float cfac[2][16];
    // of each head's warps, by query head: a block's maxima, and the sums of a piece.
    // Apart: a warp may write its sums while another still reads the maxima of the
    // piece's last block, and no barrier lies between.
    float red[2][4][16];
    float sum[2][4][16];
    int vote[2][2][4];
    int last[2];
    uint32_t tmem_base;
    int abort;
    Unit unit[2];
};

template <int kN, int kQTerms>
struct Shape {
    static constexpr int kSCols = (kN * kQTerms + 15) / 16 * 16;  // N of Q K^T
    static constexpr int kPRow = kN == 8 ? 32 : 64;               // bytes of a key's probabilities; N of P V
    static constexpr int kQTile = (kSCols + 7) / 8 * 1024;        // query terms of one head
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffP = kOffQ + 2 * kQTile;
    static constexpr int kOffShared = kOffP + 2 * kKeys * kPRow;
    static constexpr int kSmem = kOffShared + static_cast<int>(sizeof(Shared)) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    static_assert(kSCols <= 64 && kN * kPTerms <= kPRow, "columns");
};

struct SingleArgs {
    AttnArgs a;
    PlanLayout lay;
    char *ws;
    int32_t G, pairs, teams;  // pairs of kv heads; teams that the grid holds
    float sm_log2;            // sm_scale * log2(e)
};

// ------------------------------------------------------------------- the line

// Places of row t in the line: its blocks, with a selection at most K, and one
// for a row without any, which has an output too.
__device__ __forceinline__ int row_places(const AttnArgs &a, int t) {
    int r;
    const int64_t L = token_limit(a.ri, a.ri_s0, a.sl, a.sl_s0, t, a.R, a.NB, &r);
    int n = static_cast<int>((L + kKeys - 1) / kKeys);
    if (a.tk != nullptr) n = min(n, a.K);
    return max(n, 1);
}

// Pieces that the line is cut into, and where piece i begins.  A line has at most
// kPlanMaxT * kMaxNB places: 32 bits hold it times the teams.
constexpr int kLeastPlaces = 2;  // of a piece, where the line is short (16 blocks: 14.1 us with 1, 12.8 with 2, 13.5 with 4)
__device__ __forceinline__ int line_teams(int most, int total) {
    return min(most, (total + kLeastPlaces - 1) / kLeastPlaces);
}
__device__ __forceinline__ int line_begin(int i, int total, int teams) {
    return static_cast<int>(static_cast<uint32_t>(i) * static_cast<uint32_t>(total) / static_cast<uint32_t>(teams));
}

constexpr int kLineThreads = 512;

// base[t], the first place of row t, base[T] the line's length; the row in which
// each team's piece begins; the tickets and the status word zeroed.
__global__ void __launch_bounds__(kLineThreads) line_kernel(const __grid_constant__ SingleArgs t) {
    __shared__ int s_base[kPlanMaxT + 1];
    __shared__ int s_warp[kLineThreads / 32];
    const AttnArgs &a = t.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    tc::pdl_wait();
    tc::pdl_trigger();
    int32_t *base = reinterpret_cast<int32_t *>(t.ws + t.lay.gstart);
    int32_t *team_row = reinterpret_cast<int32_t *>(t.ws + t.lay.units);
    int32_t *counters = reinterpret_cast<int32_t *>(t.ws + t.lay.counters);
    for (int i = tid; i < a.T * a.Hkv; i += kLineThreads) counters[i] = 0;
    if (tid == 0) reinterpret_cast<PlanHeader *>(t.ws + t.lay.header)->status = 0;
    const int per = (a.T + kLineThreads - 1) / kLineThreads, r0 = min(a.T, tid * per), r1 = min(a.T, r0 + per);
    int sum = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = row_places(a, r);
        s_base[r] = n;
        sum += n;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    for (int r = r0; r < r1; ++r) {
        const int n = s_base[r];
        s_base[r] = at;
        base[r] = at;
        at += n;
    }
    int total = 0;
    for (int w = 0; w < kLineThreads / 32; ++w) total += s_warp[w];
    if (tid == 0) {
        s_base[a.T] = total;
        base[a.T] = total;
    }
    __syncthreads();
    const int teams = line_teams(t.teams, total);
    for (int i = tid; i < teams; i += kLineThreads) {
        const int x = line_begin(i, total, teams);
        int lo = 0, hi = a.T;  // s_base[lo] <= x < s_base[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_base[mid] <= x) lo = mid; else hi = mid;
        }
        team_row[i] = lo;
    }
}

// --------------------------------------------------------------------- waits

__device__ __forceinline__ bool aborted(Shared &sh) { return *reinterpret_cast<volatile int *>(&sh.abort) != 0; }

__device__ __forceinline__ bool wait_or_abort(Shared &sh, uint64_t *bar, uint32_t parity) {
    if (tc::mbar_wait_tries(bar, parity)) return true;
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
    return false;
}

// Warp-uniform: the warp goes on only if every lane saw the phase.
__device__ __forceinline__ bool warp_wait(Shared &sh, uint64_t *bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_tries(bar, parity));
    if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
    return ok;
}

// The 128 threads of head h's softmax, and the same with a flag of any of them.
__device__ __forceinline__ void group_sync(int h) { asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory"); }
__device__ __forceinline__ bool group_any(int h, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "bar.red.or.pred p, %1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(1 + h), "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// ------------------------------------------------------------------- softmax

// Two probabilities' terms, the lower one in the lower byte of each.
__device__ __forceinline__ void split_p(float p0, float p1, uint16_t (&t)[kPTerms]) {
#pragma unroll
    for (int k = 0; k < kPTerms; ++k) {
        t[k] = tc::f32x2_to_e4m3x2(p1, p0);
        if (k + 1 < kPTerms) {
            float a0, a1;
            tc::e4m3x2_to_f32x2(t[k], a1, a0);
            p0 = (p0 - a0) * (1 << kTermShift);
            p1 = (p1 - a1) * (1 << kTermShift);
        }
    }
}

// The query heads of one kv head as E4M3 terms in the swizzled tile `tile`
// (row term * kN + g), and what the scaling takes from their logits: 16 threads
// to a row, eight dims each.  The row is scaled by a power of two into [128,
// 256); a row with an infinity or a NaN becomes NaN, as its softmax is.
template <int kN, int kQTerms>
__device__ __forceinline__ void load_queries(const SingleArgs &t, Shared &sh, uint8_t *tile, int h, int row, int head0, int st) {
    const AttnArgs &a = t.a;
    const int d0 = (st & 15) * 8;
#pragma unroll
    for (int g = st >> 4; g < kN; g += 8) {
        const bool in = g < t.G;  // rows behind the group's heads stay as they are: columns that nobody reads
        const int64_t off = row * a.q_s0 + (head0 + g) * a.q_s1 + d0 * a.q_s2;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + off;
        if (!in) {
        } else if (a.q_s2 == 1 && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src);
            const uint32_t wp[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kQTerms == 2) {
                    x[2 * i] = __uint_as_float(wp[i] << 16);
                    x[2 * i + 1] = __uint_as_float(wp[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&wp[i]));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = load_float(a.q, a.q_dt, off + i * a.q_s2);
        }
        uint32_t top = 0;  // of magnitudes, as bits: a NaN or an infinity comes out on top
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m, 16));
        const int e = static_cast<int>(top >> 23);
        const int shift = e == 0 ? 0 : min(7 - (e - 127), 100);
        const float up = e == 255 ? NAN : __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
        if (in && (st & 15) == 0) sh.cfac[h][g] = t.sm_log2 * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= up;
#pragma unroll
        for (int k = 0; k < kQTerms; ++k) {
            uint16_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = tc::f32x2_to_e4m3x2(x[2 * i + 1], x[2 * i]);
                float hi, lo;
                tc::e4m3x2_to_f32x2(c[i], hi, lo);
                x[2 * i] -= lo;
                x[2 * i + 1] -= hi;
            }
            if (in)
                *reinterpret_cast<uint2 *>(tile + tc::swz_offset(k * kN + g, d0, 128)) =
                    make_uint2(tc::pack2x16(c[0], c[1]), tc::pack2x16(c[2], c[3]));
        }
    }
}

// The last piece of a row joins all of them: warp w takes rows w, w + 4, ...,
// a lane four dims.  Partials are read with ld.global.cg: other CTAs wrote them
// during this launch.
template <int kN>
__device__ void join_row(const SingleArgs &t, const Unit &u, int pair, int h, int st) {
    const AttnArgs &a = t.a;
    const int w = st >> 5, d4 = (st & 31) * 4;
    const float *parts = reinterpret_cast<const float *>(t.ws + t.lay.partials);
    // kRows rows at a time, kParts pieces of each in flight
    constexpr int kRows = 2, kParts = 4;
    for (int r0 = w; r0 < t.G; r0 += 4 * kRows) {
        float m[kRows], l[kRows];
        float4 o[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.f;
            o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int i0 = 0; i0 < u.n_split; i0 += kParts) {
            float2 ml[kRows][kParts];
            float4 x[kRows][kParts];
#pragma unroll
            for (int k = 0; k < kParts; ++k) {
                const int i = i0 + k;
                const int64_t cta = static_cast<int64_t>(u.team0 + i) * t.pairs + pair;
                const float *part = parts + ((cta * 2 + (i == 0 ? u.slot0 : 0)) * 2 + h) * kN * kStride;
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    const int r = r0 + 4 * j;
                    ml[j][k] = make_float2(-INFINITY, 0.f);
                    x[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < u.n_split && r < t.G) {
                        ml[j][k] = __ldcg(reinterpret_cast<const float2 *>(part + r * kStride + kD));
                        x[j][k] = __ldcg(reinterpret_cast<const float4 *>(part + r * kStride + d4));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                float top = m[j];
#pragma unroll
                for (int k = 0; k < kParts; ++k) top = fmaxf(top, ml[j][k].x);
                if (top == -INFINITY) continue;  // nothing read so far
                const float s0 = rescale(l[j], m[j] - top);
                o[j].x *= s0;
                o[j].y *= s0;
                o[j].z *= s0;
                o[j].w *= s0;
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const float s1 = rescale(ml[j][k].y, ml[j][k].x - top);  // 0 for a piece that read nothing
                    l[j] += ml[j][k].y;
                    o[j].x = fmaf(s1, x[j][k].x, o[j].x);
                    o[j].y = fmaf(s1, x[j][k].y, o[j].y);
                    o[j].z = fmaf(s1, x[j][k].z, o[j].z);
                    o[j].w = fmaf(s1, x[j][k].w, o[j].w);
                }
                m[j] = top;
            }
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = r0 + 4 * j;
            if (r >= t.G) continue;
            const float inv = l[j] != 0.f ? 1.f / l[j] : 0.f;
            __nv_bfloat16 *out = a.out + u.row * a.o_s0 + static_cast<int64_t>((2 * pair + h) * t.G + r) * a.o_s1;
            out[(d4 + 0) * a.o_s2] = __float2bfloat16_rn(o[j].x * inv);
            out[(d4 + 1) * a.o_s2] = __float2bfloat16_rn(o[j].y * inv);
            out[(d4 + 2) * a.o_s2] = __float2bfloat16_rn(o[j].z * inv);
            out[(d4 + 3) * a.o_s2] = __float2bfloat16_rn(o[j].w * inv);
        }
    }
}

template <int kN, int kQTerms>
__device__ __forceinline__ void softmax_group(const SingleArgs &t, Shared &sh, uint8_t *smem, uint32_t tmem, int h, int pair) {
    using S = Shape<kN, kQTerms>;
    const AttnArgs &a = t.a;
    const int st = threadIdx.x & (kGroup - 1), warp = st >> 5, lane = st & 31;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t col_o = tmem + lane_base + kColO + h * 64;
    uint8_t *q_tile = smem + S::kOffQ + h * S::kQTile;
    uint8_t *p_tile = smem + S::kOffP + h * kKeys * S::kPRow;
    uint32_t b = 0;  // pages so far
    float m[kN], l[kN], cf[kN];
#pragma unroll
    for (int r = 0; r < kN; ++r) m[r] = l[r] = cf[r] = 0.f;
    bool begun = false;  // the row's piece has had a page
    for (uint32_t n = 0;; ++n) {
        Unit &u = sh.unit[n & 1];
        const bool got = tc::mbar_wait_tries(&sh.u_full[n & 1], (n >> 1) & 1);
        if (!got) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        if (group_any(h, !got || aborted(sh))) return;  // together, or not at all
        const int count = u.count;
        if (count < 0) return;
        const int row = u.row, limit = u.limit;
        if (u.first) begun = false;
        if (u.first && count > 0) {  // a row without keys needs no queries
            // the last row's logits have all been read, so its queries have too
            load_queries<kN, kQTerms>(t, sh, q_tile, h, row, (2 * pair + h) * t.G, st);
            tc::fence_proxy_async();
            tc::mbar_arrive(&sh.q_full);
            group_sync(h);
#pragma unroll
            for (int r = 0; r < kN; ++r) {
                cf[r] = r < t.G ? sh.cfac[h][r] : 0.f;
                m[r] = l[r] = 0.f;
            }
        }
        for (int i = 0; i < count; ++i, ++b) {
            const int sb = b & 1;
            const int keys = limit - static_cast<int>(u.block[i]) * kKeys;  // of the page that the row reads
            const uint32_t col_s = tmem + lane_base + (2 * h + sb) * 64;
            bool have = warp_wait(sh, &sh.s_full[h][sb], (b >> 1) & 1);
            float x[kN];
#pragma unroll
            for (int r = 0; r < kN; ++r) x[r] = 0.f;
            BlockScale bs = {1.f, 0.f, 1.f};
            if (have) {
                tc::tc_fence_after();
                float v[kQTerms * kN];
#pragma unroll
                for (int c = 0; c < kQTerms * kN; c += 8) tc::tmem_ld8(col_s + c, *reinterpret_cast<float(*)[8]>(&v[c]));
                tc::tmem_wait_ld();
                bs = block_scale(sh.scale[h][b % kScaleRing]);
#pragma unroll
                for (int r = 0; r < kN; ++r) {
                    x[r] = v[r];
#pragma unroll
                    for (int k = 1; k < kQTerms; ++k) x[r] += v[k * kN + r];
                }
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&sh.s_empty[h][sb]);
            // logits in log2 units with the V scale, less the offset
            const bool valid = st < keys;
            bool over = false;
#pragma unroll
            for (int r = 0; r < kN; ++r) {
                const float z = fmaf(x[r], cf[r] * bs.k, bs.lg_v - m[r]);
                x[r] = valid ? z : -INFINITY;
                over |= x[r] > kCap;
            }
            const int mine = ((__any_sync(0xffffffffu, over) || !begun) ? 1 : 0) | ((!have || aborted(sh)) ? 2 : 0);
            if (lane == 0) sh.vote[h][sb][warp] = mine;
            group_sync(h);
            const int vote = sh.vote[h][sb][0] | sh.vote[h][sb][1] | sh.vote[h][sb][2] | sh.vote[h][sb][3];
            if (vote & 2) return;
            if (vote & 1) {
#pragma unroll
                for (int r = 0; r < kN; ++r) {
                    float top = x[r];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    if (lane == 0) sh.red[h][warp][r] = top;
                }
                group_sync(h);
                float alpha[kN];
                bool moved = false;
#pragma unroll
                for (int r = 0; r < kN; ++r) {
                    const float top = fmaxf(fmaxf(sh.red[h][0][r], sh.red[h][1][r]), fmaxf(sh.red[h][2][r], sh.red[h][3][r]));
                    // rows whose logits are all NaN have no maximum: any offset that is a
                    // number will do, and their sums stay NaN through the join
                    const float by = (top > kCap || !begun) && top > -INFINITY ? top - kTarget : 0.f;
                    alpha[r] = rescale(l[r], -by);
                    if (!begun) l[r] = 0.f;
                    moved |= by != 0.f;
                    m[r] += by;
                    x[r] -= by;
                }
                if (begun && moved) {
                    // the pages before are in O: once their last product is done, O follows
                    warp_wait(sh, &sh.pv_done[h], (b - 1) & 1);
                    tc::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kPTerms * kN; c += 8) {
                        float o[8];
                        tc::tmem_ld8(col_o + c, o);
                        tc::tmem_wait_ld();
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(o[k] * alpha[(c + k) % kN]);
                        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(col_o + c),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                     : "memory");
                    }
                    tc::tmem_wait_st();
                }
                begun = true;
            }
            uint32_t w[kPTerms][kN / 4];
#pragma unroll
            for (int r = 0; r < kN; r += 4) {
                uint16_t lo[kPTerms], hi[kPTerms];
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = tc::ex2(x[r + k]);
                    l[r + k] += tc::ex2(x[r + k] - bs.lg_v);  // not p / vs: block_scale.cuh
                }
                split_p(p[0], p[1], lo);
                split_p(p[2], p[3], hi);
#pragma unroll
                for (int k = 0; k < kPTerms; ++k) w[k][r / 4] = tc::pack2x16(lo[k], hi[k]);
            }
            // the product of the page before has read the P tile
            if (b >= 1) warp_wait(sh, &sh.pv_done[h], (b - 1) & 1);
            if (kN == 8) {
                *reinterpret_cast<uint4 *>(p_tile + tc::swz_offset(st, 0, 32)) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
                *reinterpret_cast<uint4 *>(p_tile + tc::swz_offset(st, 16, 32)) = make_uint4(w[2][0], w[2][1], 0u, 0u);
            } else {
#pragma unroll
                for (int k = 0; k < kPTerms; ++k)
                    *reinterpret_cast<uint4 *>(p_tile + tc::swz_offset(st, 16 * k, 64)) =
                        make_uint4(w[k][0], w[k][1], w[k][kN / 4 - 2], w[k][kN / 4 - 1]);
            }
            if (!valid) {
                // slots behind the row's keys may hold anything, NaN included: zeros
                wait_or_abort(sh, &sh.kv_full[b % kStages], (b / kStages) & 1);
                uint4 *v = reinterpret_cast<uint4 *>(smem + (b % kStages) * kStage + (2 + h) * kTile + st * kD);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
            }
            tc::fence_proxy_async();
            tc::tc_fence_before();
            tc::mbar_arrive(&sh.p_full[h]);
        }
        if (u.last) {
            // sums over the keys, then O, a dim to a thread
#pragma unroll
            for (int r = 0; r < kN; ++r) {
                float s = l[r];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == 0) sh.sum[h][warp][r] = s;
            }
            if (begun) warp_wait(sh, &sh.pv_done[h], (b - 1) & 1);
            tc::tc_fence_after();
            group_sync(h);
            float o[kN];
#pragma unroll
            for (int r = 0; r < kN; ++r) {
                l[r] = (sh.sum[h][0][r] + sh.sum[h][1][r]) + (sh.sum[h][2][r] + sh.sum[h][3][r]);
                o[r] = 0.f;
            }
            if (begun) {
                float v[kPTerms * kN];
#pragma unroll
                for (int c = 0; c < kPTerms * kN; c += 8) tc::tmem_ld8(col_o + c, *reinterpret_cast<float(*)[8]>(&v[c]));
                tc::tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < kN; ++r)
                    o[r] = fmaf(fmaf(v[2 * kN + r], 1.f / (1 << kTermShift), v[kN + r]), 1.f / (1 << kTermShift), v[r]);
            }
            tc::tc_fence_before();
            if (u.part < 0) {
                __nv_bfloat16 *out = a.out + row * a.o_s0 + static_cast<int64_t>((2 * pair + h) * t.G) * a.o_s1 + st * a.o_s2;
#pragma unroll
                for (int r = 0; r < kN; ++r)
                    if (r < t.G) out[r * a.o_s1] = __float2bfloat16_rn(l[r] != 0.f ? o[r] / l[r] : 0.f);
            } else {
                float *part = reinterpret_cast<float *>(t.ws + t.lay.partials) +
                              ((static_cast<int64_t>(blockIdx.x) * 2 + u.part) * 2 + h) * kN * kStride;
#pragma unroll
                for (int r = 0; r < kN; ++r) {
                    if (r >= t.G) continue;
                    part[r * kStride + st] = o[r];
                    if (st == 0) *reinterpret_cast<float2 *>(part + r * kStride + kD) = make_float2(begun ? m[r] : -INFINITY, l[r]);
                }
                __threadfence();
                group_sync(h);
                if (st == 0) {
                    int32_t *ticket = reinterpret_cast<int32_t *>(t.ws + t.lay.counters) + row * a.Hkv + 2 * pair + h;
                    sh.last[h] = atomicAdd(ticket, 1) == u.n_split - 1;
                }
                group_sync(h);
                if (sh.last[h]) {
                    __threadfence();
                    join_row<kN>(t, u, pair, h, st);
                }
            }
            group_sync(h);  // the sums and the ticket before they are written again
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.u_empty[n & 1]);
    }
}

template <int kN, int kQTerms>
__global__ void __launch_bounds__(kThreads, 1)
attention_single_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ SingleArgs t) {
    using S = Shape<kN, kQTerms>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared &sh = *reinterpret_cast<Shared *>(smem + S::kOffShared);
    const AttnArgs &a = t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = blockIdx.x / t.pairs, pair = blockIdx.x % t.pairs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.u_full[i], 1);
            tc::mbar_init(&sh.u_empty[i], kUnitReleases);
            tc::mbar_init(&sh.p_full[i], kGroup);
            tc::mbar_init(&sh.pv_done[i], 1);
            tc::mbar_init(&sh.drain[i], 1);
            for (int k = 0; k < 2; ++k) {
                tc::mbar_init(&sh.s_full[i][k], 1);
                tc::mbar_init(&sh.s_empty[i][k], kGroup);
            }
        }
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&sh.kv_full[i], 3);   // the copies, and both heads' scales
            tc::mbar_init(&sh.kv_empty[i], 2);  // both issuers
        }
        tc::mbar_init(&sh.q_full, 2 * kGroup);
        sh.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kWarpQk) tc::tmem_alloc(&sh.tmem_base, kTmemCols);
    if (threadIdx.x == kWarpPv * 32) {
        tc::prefetch_tmap(&tmap_k);
        tc::prefetch_tmap(&tmap_v);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    tc::pdl_wait();  // the line
    tc::pdl_trigger();

    if (warp >= kWarpSoft) {
        softmax_group<kN, kQTerms>(t, sh, smem, tmem, (warp - kWarpSoft) >> 2, pair);
    } else if (warp == kWarpTma) {
        if (lane == 0) {
            // pages are read once (16 x 16384 keys 87.0 us, without the hint 88.8; rows
            // that share selected pages 22.9 and 24.4)
            const uint64_t policy = tc::policy_evict_first();
            uint32_t b = 0;
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                Unit &u = sh.unit[n & 1];
                ok = wait_or_abort(sh, &sh.u_full[n & 1], (n >> 1) & 1);
                if (!ok || u.count < 0) break;
                const int count = u.count;
                for (int i = 0; i < count; ++i, ++b) {
                    const int st = b % kStages;
                    if (aborted(sh) || (b >= kStages && !wait_or_abort(sh, &sh.kv_empty[st], (b / kStages - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    const int page = u.page[i];
                    uint8_t *at = smem + st * kStage;
                    tc::mbar_arrive_expect_tx(&sh.kv_full[st], kStage);
                    for (int h = 0; h < 2; ++h)
                        tc::tma_load_3d(at + h * kTile, &tmap_k, &sh.kv_full[st], 0, 2 * pair + h, page * kKeys, policy);
                    for (int h = 0; h < 2; ++h)
                        tc::tma_load_3d(at + (2 + h) * kTile, &tmap_v, &sh.kv_full[st], 0, 2 * pair + h, page * kKeys, policy);
                    for (int h = 0; h < 2; ++h)
                        load_block_scale(&sh.scale[h][b % kScaleRing], a.sc, page, 2 * pair + h, &sh.kv_full[st]);
                }
                if (ok) tc::mbar_arrive(&sh.u_empty[n & 1]);
            }
            // every issued copy lands before the CTA may exit
            for (uint32_t k = b > kStages ? b - kStages : 0; k < b; ++k) tc::mbar_wait_tries(&sh.kv_full[k % kStages], (k / kStages) & 1);
        }
    } else if (warp == kWarpQk) {
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_m128(S::kSCols, false, false);
            const uint64_t dk0 = tc::smem_desc(tc::smem_u32(smem), 16, 1024, tc::kSw128);
            const uint64_t dq0 = tc::smem_desc(tc::smem_u32(smem + S::kOffQ), 16, 1024, tc::kSw128);
            uint32_t b = 0, nq = 0;
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                Unit &u = sh.unit[n & 1];
                ok = wait_or_abort(sh, &sh.u_full[n & 1], (n >> 1) & 1);
                if (!ok || u.count < 0) break;
                const int count = u.count;
                if (u.first && count > 0) {
                    ok = wait_or_abort(sh, &sh.q_full, nq & 1);
                    if (!ok) break;
                    ++nq;
                }
                for (int i = 0; i < count; ++i, ++b) {
                    const int st = b % kStages, sb = b & 1;
                    ok = wait_or_abort(sh, &sh.kv_full[st], (b / kStages) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (b >= 2 && !wait_or_abort(sh, &sh.s_empty[h][sb], ((b >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc::tc_fence_after();
                        const uint64_t dk = dk0 + ((st * kStage + h * kTile) >> 4), dq = dq0 + ((h * S::kQTile) >> 4);
#pragma unroll
                        for (int ks = 0; ks < kD / 32; ++ks)  // 32 dims, 32 bytes into the rows
                            tc::mma_f8(tmem + (2 * h + sb) * 64, dk + 2 * ks, dq + 2 * ks, idesc, ks > 0);
                        tc::mma_commit(&sh.s_full[h][sb]);
                    }
                    if (!ok) break;
                    tc::mma_commit(&sh.kv_empty[st]);
                }
                if (ok) tc::mbar_arrive(&sh.u_empty[n & 1]);
            }
            // every issued product completes before tensor memory is released
            tc::mma_commit(&sh.drain[0]);
            tc::mbar_wait_tries(&sh.drain[0], 0);
        }
    } else if (warp == kWarpPv) {
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_m128(S::kPRow, true, true);
            const uint64_t dv0 = tc::smem_desc(tc::smem_u32(smem), kTile, 1024, tc::kSw128);
            const uint64_t dp0 = tc::smem_desc(tc::smem_u32(smem + S::kOffP), kKeys * S::kPRow, 8 * S::kPRow,
                                               S::kPRow == 32 ? tc::kSw32 : tc::kSw64);
            uint32_t b = 0;
            bool ok = true, begun = false;
            for (uint32_t n = 0; ok; ++n) {
                Unit &u = sh.unit[n & 1];
                ok = wait_or_abort(sh, &sh.u_full[n & 1], (n >> 1) & 1);
                if (!ok || u.count < 0) break;
                const int count = u.count;
                if (u.first) begun = false;
                for (int i = 0; i < count; ++i, ++b) {
                    const int st = b % kStages;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // P, and behind a row's first one the last row's O has been read
                        if (!wait_or_abort(sh, &sh.p_full[h], b & 1)) {
                            ok = false;
                            break;
                        }
                        tc::tc_fence_after();
                        const uint64_t dv = dv0 + ((st * kStage + (2 + h) * kTile) >> 4), dp = dp0 + ((h * kKeys * S::kPRow) >> 4);
#pragma unroll
                        for (int ks = 0; ks < kKeys / 32; ++ks)  // 32 keys
                            tc::mma_f8(tmem + kColO + h * 64, dv + ks * (32 * kD >> 4), dp + ks * (32 * S::kPRow >> 4), idesc,
                                       begun || ks > 0);
                        tc::mma_commit(&sh.pv_done[h]);
                    }
                    if (!ok) break;
                    tc::mma_commit(&sh.kv_empty[st]);
                    begun = true;
                }
                if (ok) tc::mbar_arrive(&sh.u_empty[n & 1]);
            }
            tc::mma_commit(&sh.drain[1]);
            tc::mbar_wait_tries(&sh.drain[1], 0);
        }
    } else {
        // ------------------------------------------------------- block lists
        const int32_t *base = reinterpret_cast<const int32_t *>(t.ws + t.lay.gstart);
        const int total = base[a.T], teams = line_teams(t.teams, total);
        auto begin_of = [&](int i) { return line_begin(i, total, teams); };
        auto team_of = [&](int x) { return static_cast<int>((static_cast<uint32_t>(x + 1) * teams - 1) / total); };
        int x = 0, x1 = 0, row = 0;
        if (team < teams) {
            x = begin_of(team);
            x1 = begin_of(team + 1);
            row = reinterpret_cast<const int32_t *>(t.ws + t.lay.units)[team];
        }
        const int row0 = row;
        uint32_t n = 0;
        bool ok = true;
        auto claim = [&] { return n < 2 || warp_wait(sh, &sh.u_empty[n & 1], ((n >> 1) - 1) & 1); };
        for (; x < x1 && ok; ++row) {
            const int base_t = base[row], end_t = base[row + 1];
            int r;
            const int64_t L = token_limit(a.ri, a.ri_s0, a.sl, a.sl_s0, row, a.R, a.NB, &r);
            const int vis = static_cast<int>((L + kKeys - 1) / kKeys);
            const int lo = x - base_t, hi = min(x1, end_t) - base_t;  // ranks of the row's list
            // lane l holds blocks 32 l ..
            uint32_t word = lane * 32 >= vis ? 0u : (vis - lane * 32 >= 32 ? 0xffffffffu : (1u << (vis - lane * 32)) - 1u);
            ok = claim() && !aborted(sh);
            if (!ok) break;
            Unit *u = &sh.unit[n & 1];
            if (a.tk != nullptr) {
                // the selection as a set, in the unit's own list space
                uint32_t *bits = reinterpret_cast<uint32_t *>(u->page);
                bits[lane] = 0;
                __syncwarp();
                for (int k = lane; k < a.K; k += 32) {
                    const int id = a.tk[row * a.tk_s1 + k * a.tk_s2];
                    if (id >= 0 && id < a.NB) atomicOr(&bits[id >> 5], 1u << (id & 31));
                }
                __syncwarp();
                word &= bits[lane];
                __syncwarp();
            }
            int before = __popc(word);
            const int mine = before;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, d);
                if (lane >= d) before += y;
            }
            before -= mine;
            int count = 0, first = 1;
            auto publish = [&](int last) {
                if (lane == 0) {
                    u->count = count;
                    u->row = row;
                    u->limit = static_cast<int32_t>(L);
                    u->first = first;
                    u->last = last;
                    const int i0 = team_of(base_t), i1 = team_of(end_t - 1);
                    u->part = i0 == i1 ? -1 : (row == row0 ? 0 : 1);
                    u->team0 = i0;
                    u->n_split = i1 - i0 + 1;
                    u->slot0 = begin_of(i0) >= base_t ? 0 : 1;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.u_full[n & 1]);
                ++n;
            };
            for (int w = 0; w * 32 < vis; ++w) {
                const uint32_t ww = __shfl_sync(0xffffffffu, word, w);
                const int wb = __shfl_sync(0xffffffffu, before, w);
                if (wb >= hi || wb + __popc(ww) <= lo) continue;
                const int rank = wb + __popc(ww & ((1u << lane) - 1u));
                bool take = ((ww >> lane) & 1u) && rank >= lo && rank < hi;
                int32_t page = -1;
                if (take) page = a.bt[r * a.bt_s0 + (w * 32 + lane) * a.bt_s1];
                take = take && page >= 0 && page < a.P;
                const uint32_t taken = __ballot_sync(0xffffffffu, take);
                if (count + __popc(taken) > kListCap) {
                    publish(0);
                    ok = claim() && !aborted(sh);
                    if (!ok) break;
                    u = &sh.unit[n & 1];
                    count = 0;
                    first = 0;
                }
                if (take) {
                    const int at = count + __popc(taken & ((1u << lane) - 1u));
                    u->page[at] = page;
                    u->block[at] = static_cast<uint16_t>(w * 32 + lane);
                }
                count += __popc(taken);
            }
            if (!ok) break;
            publish(1);
            x = base_t + hi;
        }
        if (ok && claim()) {
            if (lane == 0) {
                sh.unit[n & 1].count = -1;
                tc::mbar_arrive(&sh.u_full[n & 1]);
            }
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (threadIdx.x == 0 && aborted(sh)) atomicOr(&reinterpret_cast<PlanHeader *>(t.ws + t.lay.header)->status, 1);
    if (warp == kWarpQk) tc::tmem_dealloc(tmem, kTmemCols);
}

// E4M3 cache [slots, Hkv, 128 bytes] as a 3-D map whose box is 128 slots of one
// kv head, 128-byte swizzle.
bool make_map(CUtensorMap *m, const uint8_t *base, int64_t slots, int64_t hkv, int64_t s0, int64_t s1) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(hkv), static_cast<cuuint64_t>(slots)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s0)};
    cuuint32_t box[3] = {kD, 1, kKeys};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_pdl(const void *func, int grid, int threads, int smem, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, func, args);
}

template <int kN, int kQTerms>
cudaError_t launch(SingleArgs &t, CUtensorMap &mk, CUtensorMap &mv, cudaStream_t stream) {
    const void *func = reinterpret_cast<const void *>(attention_single_kernel<kN, kQTerms>);
    cudaError_t e = opt_in_smem(func, Shape<kN, kQTerms>::kSmem);
    if (e != cudaSuccess) return e;
    void *line_args[] = {&t};
    e = launch_pdl(reinterpret_cast<const void *>(line_kernel), 1, kLineThreads, 0, line_args, stream);
    if (e != cudaSuccess) return e;
    void *args[] = {&mk, &mv, &t};
    return launch_pdl(func, t.teams * t.pairs, kThreads, Shape<kN, kQTerms>::kSmem, args, stream);
}

}  // namespace

// Covers block-scaled E4M3 caches with 16-byte aligned rows of 128 dims, bf16 or
// f16 queries, an even number of kv heads up to 64 that share one selection, at
// most 4096 rows, page tables of up to 1024 blocks.  Anything else: *used stays
// false.
cudaError_t launch_attention_single(const AttnArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream, bool *used) {
    *used = false;
    const int G = a.Hq / a.Hkv;
    if (a.sc.k == nullptr || a.kv_dt != SPD_E4M3 || a.D != kD || (a.q_dt != SPD_BF16 && a.q_dt != SPD_F16)) return cudaSuccess;
    if (a.Hkv % 2 != 0 || a.Hkv > 64 || G < 1 || G > 16 || a.T > kPlanMaxT || a.NB > kMaxNB) return cudaSuccess;
    if (a.tk != nullptr && a.tk_s0 != 0) return cudaSuccess;
    if ((a.k_s0 % 16) || (a.k_s1 % 16) || (a.v_s0 % 16) || (a.v_s1 % 16)) return cudaSuccess;
    if ((reinterpret_cast<uintptr_t>(a.k) % 16) || (reinterpret_cast<uintptr_t>(a.v) % 16)) return cudaSuccess;
    if (a.P < 1 || a.P * kKeys > (int64_t(1) << 31) - 1) return cudaSuccess;
    SingleArgs t{};
    t.lay = PlanLayout(a.T, a.Hq, a.Hkv, a.D, a.NB);
    if (ws == nullptr || ws_bytes < t.lay.total) return cudaSuccess;
    t.a = a;
    t.ws = static_cast<char *>(ws);
    t.G = G;
    t.pairs = a.Hkv / 2;
    t.teams = std::max(1, device_sm_count() / t.pairs);
    t.sm_log2 = a.sm_scale * 1.4426950408889634f;
    const int n = G <= 8 ? 8 : 16;
    // two partial rows' slots of a CTA, two heads each, and a word a team
    if (static_cast<int64_t>(t.teams) * t.pairs * 4 * n > t.lay.rows_cap || t.teams > t.lay.unit_cap || t.teams > 1000)
        return cudaSuccess;
    CUtensorMap mk, mv;
    if (!make_map(&mk, a.k, a.P * kKeys, a.Hkv, a.k_s0, a.k_s1) || !make_map(&mv, a.v, a.P * kKeys, a.Hkv, a.v_s0, a.v_s1))
        return cudaSuccess;
    const bool bf16 = a.q_dt == SPD_BF16;
    const cudaError_t e = n == 8 ? (bf16 ? launch<8, 2>(t, mk, mv, stream) : launch<8, 3>(t, mk, mv, stream))
                                 : (bf16 ? launch<16, 2>(t, mk, mv, stream) : launch<16, 3>(t, mk, mv, stream));
    if (e == cudaSuccess) *used = true;
    return e;
}

}  // namespace spd
