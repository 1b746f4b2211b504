// chunk_plan.cu -- device planner of the tensor-core prefill attention.
//
// CTA 0 works through the batch in four steps, all sums in shared memory:
// sequences are ranked by the keys they read (longest first: the units that
// are claimed last are then the short ones), cut into pairs, a piece length is
// chosen for the whole batch, and the pairs get their unit and partial ranges.
//
// The piece length: N CTAs claim the units in order, longest about first.  The
// unit at place i * N then starts when some CTA has done i others at least as
// long, so cutting the costs into pieces of at most U blocks takes no less than
//   max over i of (i + 1) * (length of the unit at place i * N + o)
// block times, nor than the work and the units' own costs shared evenly; o =
// kUnitBlocks is what a unit costs beside its blocks (first loads, epilogue,
// partials).  The larger of the two is the estimate: over drawn batches the
// piece length it picks runs within 1 % of the best one's simulated time (40 %
// at worst, on batches of a few short units).  U = ceil(max c / m) for m =
// 1 .. kMaxPieces is tried, a value to a warp at a time, and the smallest
// estimate whose split pieces fit the partial slots is taken (ties to longer
// pieces).  Finer pieces than make kWaves units a CTA are not tried: a batch of
// hundreds of pairs has nothing left to even out.  The search multiplies by
// reciprocals; integer divisions took half of the plan's 12 us (8 chunks of
// 512 tokens: 12.3 -> 6.5 us).
// Everything depends on the lengths alone, so equal batches are always cut,
// and joined, alike.
#include "chunk_plan.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"
#include "tc_ptx.cuh"

namespace spd {

namespace {

constexpr int kPlanT = 512;
constexpr int kPlanWarps = kPlanT / 32;
constexpr int kMaxRanked = 1024;  // sequences that are ordered by length (each is compared with each)
constexpr int kSmemPairs = 2048;  // pairs whose lengths and places fit shared memory
constexpr int kMaxPieces = 64;
constexpr int kWaves = 16;        // units beyond this many a CTA are not cut finer
constexpr float kUnitBlocks = 3.f;

// Exclusive prefix sum over the CTA and the total.
__device__ __forceinline__ int32_t scan_cta(int32_t x, int32_t *sums, int32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int32_t w = lane < kPlanWarps ? sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return incl - x + (warp > 0 ? before : 0);
}

// Everything the steps share lies in shared memory: the batch's metadata is
// read once, the pair records are written once, and between the two no step
// waits for global memory.  (Batches of more than kSmemPairs pairs keep the
// two arrays that a pair has in the workspace instead.)
__device__ void plan_batch(const ChunkPlanArgs &p) {
    extern __shared__ int32_t dyn[];
    __shared__ int32_t sums[32];
    __shared__ int32_t small[2 * kSmemPairs];
    __shared__ float best_est[kPlanWarps];
    __shared__ int32_t best_u[kPlanWarps];
    __shared__ int32_t cmax_s;
    const ChunkArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ChunkHeader *hd = reinterpret_cast<ChunkHeader *>(p.ws + p.lay.header);
    ChunkPair *pairs = reinterpret_cast<ChunkPair *>(p.ws + p.lay.pairs);
    ChunkSplit *splits = reinterpret_cast<ChunkSplit *>(p.ws + p.lay.splits);
    // per sequence: first token, tokens, cached keys, keys in all; order by
    // length, and pair offsets in that order
    int32_t *start = dyn, *n_tok = start + a.B, *pre = n_tok + a.B, *cap = pre + a.B, *order = cap + a.B, *poff = order + a.B;
    const int pair_tokens = 2 * p.lay.tt;

    for (int b = tid; b < a.B; b += kPlanT) {
        const int32_t lo = min(max(a.cu[b * a.cu_s0], 0), a.total_q);
        const int32_t hi = min(max(a.cu[(b + 1) * a.cu_s0], 0), a.total_q);
        const int32_t r = a.sid[b * a.sid_s0];
        start[b] = lo;
        n_tok[b] = max(hi - lo, 0);
        pre[b] = min(max(a.pre[b * a.pre_s0], -(1 << 30)), 1 << 30);
        cap[b] = r >= 0 && r < a.R ? min(a.sl[b * a.sl_s0], a.NB * kBlock) : 0;
    }
    if (tid == 0) cmax_s = 0;
    __syncthreads();
    auto limit = [&](int b, int32_t i) { return max(min(pre[b] + i + 1, cap[b]), 0); };

    // order of the sequences: by keys read, descending, ties by index
    if (a.B <= kMaxRanked) {
        for (int b = tid; b < a.B; b += kPlanT) poff[b] = n_tok[b] > 0 ? limit(b, n_tok[b] - 1) : -1;
        __syncthreads();
        for (int b = tid; b < a.B; b += kPlanT) {
            const int32_t mine = poff[b];
            int rank = 0;
#pragma unroll 4
            for (int o = 0; o < a.B; ++o) rank += poff[o] > mine || (poff[o] == mine && o < b);
            order[rank] = b;
        }
    } else {
        for (int b = tid; b < a.B; b += kPlanT) order[b] = b;
    }
    __syncthreads();

    // pairs of each sequence, in that order
    int32_t carry = 0;
    for (int base = 0; base < a.B; base += kPlanT) {
        const int k = base + tid;
        int32_t np = 0, total;
        if (k < a.B) np = (n_tok[order[k]] + pair_tokens - 1) / pair_tokens;
        const int32_t at = scan_cta(np, sums, &total);
        if (k < a.B) poff[k] = carry + at;
        carry += total;
    }
    if (tid == 0) poff[a.B] = carry;
    __syncthreads();
    // offsets that decrease could name more pairs than the workspace holds
    const int32_t n_pairs = static_cast<int32_t>(min(static_cast<int64_t>(carry), p.lay.pair_cap));
    int32_t *costs = n_pairs <= kSmemPairs ? small : reinterpret_cast<int32_t *>(p.ws + p.lay.pair_tmp);
    int32_t *unit0 = n_pairs <= kSmemPairs ? small + kSmemPairs : costs + p.lay.pair_cap;
    // the place of pair q in the order, and its first token and tokens there
    auto place = [&](int q, int32_t &i0, int32_t &nt) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (poff[mid] <= q) lo = mid; else hi = mid;
        }
        const int32_t n = n_tok[order[lo]];
        const int64_t at = (static_cast<int64_t>(q) - poff[lo]) * pair_tokens;
        const bool inside = at >= 0 && at < n;  // always, unless the offsets decrease
        i0 = inside ? static_cast<int32_t>(at) : 0;
        nt = inside ? min(pair_tokens, n - i0) : 0;
        return lo;
    };
    int32_t cmax = 0;
    for (int q = tid; q < n_pairs; q += kPlanT) {
        int32_t i0, nt;
        const int b = order[place(q, i0, nt)];
        int64_t cost = nt > 0 ? (limit(b, i0 + nt - 1) + kBlock - 1) / kBlock : 0;
        if (a.tk != nullptr && nt > 0) {
            // each tile takes the blocks that its query blocks list, at most
            // all that there are; two tiles side by side
            const int32_t nt0 = min(nt, p.lay.tt);
            const int64_t c0 = min(cost, static_cast<int64_t>((i0 + nt0 - 1) / a.bsq - i0 / a.bsq + 1) * a.K);
            const int64_t c1 = min(cost, static_cast<int64_t>((i0 + nt - 1) / a.bsq - (i0 + nt0) / a.bsq + 1) * a.K);
            cost = nt > nt0 ? (c0 + c1 + 1) / 2 : c0;
        }
        // one tile of rows: two pages at a time, for a little more than one
        if (nt <= p.lay.tt) cost = (3 * cost + 4) / 5;
        costs[q] = static_cast<int32_t>(cost);
        cmax = max(cmax, static_cast<int32_t>(cost));
    }
    cmax = __reduce_max_sync(0xffffffffu, cmax);
    if (lane == 0) atomicMax(&cmax_s, cmax);
    __syncthreads();
    cmax = max(cmax_s, 1);

    // pieces of a pair of cost c at most U long; by the reciprocal of U, exact
    // while c + U stays below 2^21 (c is at most the table's kMaxNB)
    auto cut = [](int32_t c, int32_t U, float inv) {
        return max(static_cast<int32_t>((static_cast<float>(c + U - 1) + 0.5f) * inv), 1);
    };
    // piece length: a batch of many units gains little from more
    const float inv_ctas = 1.f / static_cast<float>(p.ctas);
    const int m_max = min(max(kWaves * p.ctas / max(n_pairs * a.Hkv, 1), 1), kMaxPieces);
    float est_best = INFINITY;
    int32_t u_best = cmax;
    for (int m = warp + 1; m <= m_max; m += kPlanWarps) {
        const int32_t U = (cmax + m - 1) / m;
        const float inv = 1.f / static_cast<float>(U);
        int32_t units = 0;
        float parts = 0.f, work = 0.f, longest = 0.f;
        for (int base = 0; base < n_pairs; base += 32) {
            const int q = base + lane;
            const int32_t c = q < n_pairs ? costs[q] : 0;
            const int32_t k = q < n_pairs ? cut(c, U, inv) : 0;
            int32_t incl = k;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            // the last multiple of N among the places of the pair's units
            const int32_t end = (units + incl) * a.Hkv;
            const int32_t i = static_cast<int32_t>((static_cast<float>(end - 1) + 0.5f) * inv_ctas);
            if (k > 0 && i * p.ctas >= end - k * a.Hkv)
                longest = fmaxf(longest, static_cast<float>(i + 1) *
                                             (floorf(__fdividef(static_cast<float>(c + k) - 0.5f, static_cast<float>(k))) + kUnitBlocks));
            units += __shfl_sync(0xffffffffu, incl, 31);
            parts += k > 1 ? static_cast<float>(k) : 0.f;
            work += static_cast<float>(c);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            parts += __shfl_xor_sync(0xffffffffu, parts, d);
            work += __shfl_xor_sync(0xffffffffu, work, d);
            longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, d));
        }
        const float heads = static_cast<float>(a.Hkv);
        const float est = fmaxf(longest, heads * (work + kUnitBlocks * static_cast<float>(units)) * inv_ctas);
        if (parts * heads <= static_cast<float>(p.lay.part_cap) && est < est_best) {
            est_best = est;
            u_best = U;
        }
    }
    if (lane == 0) {
        best_est[warp] = est_best;
        best_u[warp] = u_best;
    }
    __syncthreads();
    float e = lane < kPlanWarps ? best_est[lane] : INFINITY;
    int32_t U = lane < kPlanWarps ? best_u[lane] : cmax;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float oe = __shfl_xor_sync(0xffffffffu, e, d);
        const int32_t ou = __shfl_xor_sync(0xffffffffu, U, d);
        if (oe < e || (oe == e && ou > U)) {
            e = oe;
            U = ou;
        }
    }

    // unit ranges, then the records
    const float inv_u = 1.f / static_cast<float>(U);
    auto pieces_of = [&](int q) { return cut(costs[q], U, inv_u); };
    int32_t ucarry = 0;
    for (int base = 0; base < n_pairs; base += kPlanT) {
        const int q = base + tid;
        int32_t total;
        const int32_t at = scan_cta(q < n_pairs ? pieces_of(q) : 0, sums, &total);
        if (q < n_pairs) unit0[q] = ucarry + at;
        ucarry += total;
    }
    __syncthreads();
    int32_t pcarry = 0, scarry = 0;
    for (int base = 0; base < n_pairs; base += kPlanT) {
        const int q = base + tid;
        const int32_t k = q < n_pairs ? pieces_of(q) : 0;
        int32_t ptotal, stotal;
        const int32_t kp = scan_cta(k > 1 ? k : 0, sums, &ptotal);
        const int32_t ks = scan_cta(k > 1 ? 1 : 0, sums, &stotal);
        if (q < n_pairs) {
            ChunkPair r;
            const int at = place(q, r.i0, r.nt);
            r.b = order[at];
            r.tok0 = start[r.b] + r.i0;
            r.key.unit0 = unit0[q];
            r.key.pieces = k;
            r.key.seq0 = unit0[min(max(poff[at], 0), n_pairs - 1)];
            r.key.seq_units = (poff[at + 1] < n_pairs ? unit0[max(poff[at + 1], 0)] : ucarry) - r.key.seq0;
            r.part0 = pcarry + kp;
            r.row = a.sid[r.b * a.sid_s0];
            r.pre = pre[r.b];
            r.cap = cap[r.b];
            pairs[q] = r;
            if (k > 1) *reinterpret_cast<int4 *>(&splits[scarry + ks]) = make_int4(r.tok0, r.nt, k, r.part0);
        }
        pcarry += ptotal;
        scarry += stotal;
    }
    if (tid == 0) {
        hd->status = 0;
        hd->next_unit = 0;
        hd->n_pairs = n_pairs;
        hd->n_units = ucarry * a.Hkv;
        hd->head_parts = pcarry;
        hd->n_splits = scarry;
    }
}

__global__ void __launch_bounds__(kPlanT) chunk_plan_kernel(const __grid_constant__ ChunkPlanArgs p) {
    // the attention kernel may take the free SMs and set itself up; it waits
    // for this kernel's end before it reads global memory (sparse bf16, 1111
    // tokens, 67.5 -> 62.0 us; sparse E4M3, 4096 tokens, 344 -> 346)
    tc::pdl_trigger();
    if (blockIdx.x == 0) {
        plan_batch(p);
        return;
    }
    const ChunkArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t gwarp = (static_cast<int64_t>(blockIdx.x - 1) * kPlanT + threadIdx.x) / 32;
    const int64_t n_warps = static_cast<int64_t>(gridDim.x - 1) * kPlanWarps;

    // selection rows to bitmaps of key blocks, one warp a row
    if (a.tk != nullptr) {
        __shared__ uint32_t words[kPlanWarps][kMaxNB / 32];
        uint32_t *w = words[threadIdx.x >> 5];
        uint32_t *bm = reinterpret_cast<uint32_t *>(p.ws + p.lay.bitmaps);
        const int64_t rows = static_cast<int64_t>(p.heads_built) * a.n_rows;
        for (int64_t r = gwarp; r < rows; r += n_warps) {
            w[lane] = 0;
            __syncwarp();
            const int32_t *ids = a.tk + (r / a.n_rows) * a.tk_s0 + (r % a.n_rows) * a.tk_s1;
            for (int k = lane; k < a.K; k += 32) {
                const int32_t id = ids[k * a.tk_s2];
                if (id >= 0 && id < a.NB) atomicOr(&w[id >> 5], 1u << (id & 31));
            }
            __syncwarp();
            if (lane < p.lay.words) bm[r * p.lay.words + lane] = w[lane];
            __syncwarp();
        }
    }

    // output rows of tokens in front of the first and behind the last sequence
    const int32_t front = a.B > 0 ? min(max(a.cu[0], 0), a.total_q) : 0;
    const int32_t back = a.B > 0 ? min(max(a.cu[a.B * a.cu_s0], 0), a.total_q) : 0;
    const int64_t row_cells = static_cast<int64_t>(a.Hq) * a.D;
    for (int64_t k = gwarp; k < static_cast<int64_t>(front) + (a.total_q - back); k += n_warps) {
        const int64_t t = k < front ? k : back + (k - front);
        for (int64_t c = lane; c < row_cells; c += 32)
            static_cast<__nv_bfloat16 *>(a.out)[t * a.o_s0 + (c / a.D) * a.o_s1 + (c % a.D) * a.o_s2] =
                __float2bfloat16_rn(0.f);
    }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkPlanArgs &p, cudaStream_t stream) {
    const int bytes = (6 * p.a.B + 1) * static_cast<int>(sizeof(int32_t));
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(chunk_plan_kernel), bytes);
    if (e != cudaSuccess) return e;
    // beside the planning CTA, one for about every 32 selection rows, or 64
    // output rows that may have to be zeroed
    int64_t others = (static_cast<int64_t>(p.a.total_q) + 63) / 64;
    if (p.a.tk != nullptr) others += (static_cast<int64_t>(p.heads_built) * p.a.n_rows + 31) / 32;
    const int64_t most = device_sm_count() > 1 ? device_sm_count() - 1 : 1;
    chunk_plan_kernel<<<static_cast<unsigned>(1 + (others < most ? others : most)), kPlanT, bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace spd
