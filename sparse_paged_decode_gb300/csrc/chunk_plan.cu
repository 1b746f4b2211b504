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
// 1 .. kMaxPieces is tried, two values to a warp, and the smallest estimate
// whose split pieces fit the partial slots is taken (ties to longer pieces).
// Everything depends on the lengths alone, so equal batches are always cut,
// and joined, alike.
#include "chunk_plan.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"

namespace spd {

namespace {

constexpr int kPlanT = 1024;
constexpr int kMaxRanked = 1024;  // sequences that are ordered by length
constexpr int kMaxPieces = 64;
constexpr float kUnitBlocks = 3.f;

struct Seq {
    int32_t n, limit;  // tokens, and keys its last token reads
};

// Tokens of sequence b (offsets clipped to the batch).
__device__ __forceinline__ int32_t seq_tokens(const ChunkArgs &a, int b, int32_t *start) {
    const int32_t lo = min(max(a.cu[b * a.cu_s0], 0), a.total_q);
    const int32_t hi = min(max(a.cu[(b + 1) * a.cu_s0], 0), a.total_q);
    *start = lo;
    return max(hi - lo, 0);
}

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
    int32_t w = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return incl - x + (warp > 0 ? before : 0);
}

__device__ void plan_batch(const ChunkPlanArgs &p) {
    extern __shared__ int32_t dyn[];  // order [B], pair offsets in that order [B + 1]
    __shared__ int32_t sums[32];
    __shared__ int32_t limits[kMaxRanked];
    __shared__ float best_est[32];
    __shared__ int32_t best_u[32];
    __shared__ int32_t cmax_s;
    const ChunkArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ChunkHeader *hd = reinterpret_cast<ChunkHeader *>(p.ws + p.lay.header);
    ChunkPair *pairs = reinterpret_cast<ChunkPair *>(p.ws + p.lay.pairs);
    int32_t *order = dyn, *poff = dyn + a.B;
    const int pair_tokens = 2 * p.lay.tt;

    // order of the sequences: by keys read, descending, ties by index
    if (a.B <= kMaxRanked) {
        int32_t mine = 0;
        if (tid < a.B) {
            int32_t start;
            const int32_t n = seq_tokens(a, tid, &start);
            mine = n > 0 ? chunk_limit(a, tid, n - 1) : -1;
            limits[tid] = mine;
        }
        __syncthreads();
        if (tid < a.B) {
            int rank = 0;
            for (int o = 0; o < a.B; ++o) rank += limits[o] > mine || (limits[o] == mine && o < tid);
            order[rank] = tid;
        }
    } else {
        for (int b = tid; b < a.B; b += kPlanT) order[b] = b;
    }
    __syncthreads();

    // pairs of each sequence, in that order
    int32_t carry = 0;
    for (int base = 0; base < a.B; base += kPlanT) {
        const int k = base + tid;
        int32_t np = 0, start, total;
        if (k < a.B) np = (seq_tokens(a, order[k], &start) + pair_tokens - 1) / pair_tokens;
        const int32_t at = scan_cta(np, sums, &total);
        if (k < a.B) poff[k] = carry + at;
        carry += total;
    }
    if (tid == 0) {
        poff[a.B] = carry;
        cmax_s = 0;
    }
    __syncthreads();
    // offsets that decrease could name more pairs than the workspace holds
    const int32_t n_pairs = min(static_cast<int64_t>(carry), p.lay.pair_cap);
    int32_t cmax = 0;
    for (int q = tid; q < n_pairs; q += kPlanT) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (poff[mid] <= q) lo = mid; else hi = mid;
        }
        const int b = order[lo];
        int32_t start;
        const int32_t n = seq_tokens(a, b, &start);
        ChunkPair r;
        r.b = b;
        const int64_t i0 = (static_cast<int64_t>(q) - poff[lo]) * pair_tokens;
        const bool inside = i0 >= 0 && i0 < n;  // always, unless the offsets decrease
        r.i0 = inside ? static_cast<int32_t>(i0) : 0;
        r.nt = inside ? min(pair_tokens, n - r.i0) : 0;
        r.tok0 = start + r.i0;
        int64_t cost = r.nt > 0 ? (chunk_limit(a, b, r.i0 + r.nt - 1) + kBlock - 1) / kBlock : 0;
        if (a.tk != nullptr) {
            const int64_t rows = (r.i0 + r.nt - 1) / a.bsq - r.i0 / a.bsq + 1;
            cost = min(cost, rows * a.K);
        }
        r.cost = static_cast<int32_t>(cost);
        r.unit0 = r.pieces = r.part0 = 0;
        r.seq0 = poff[lo];  // for now the pair indexes that the sequence spans
        r.seq_units = min(poff[lo + 1], n_pairs);
        r.reserved[0] = r.reserved[1] = 0;
        pairs[q] = r;
        cmax = max(cmax, r.cost);
    }
    cmax = __reduce_max_sync(0xffffffffu, cmax);
    if (lane == 0) atomicMax(&cmax_s, cmax);
    __syncthreads();  // pairs are read below by other threads of this CTA only
    cmax = max(cmax_s, 1);

    // piece length
    float est_best = INFINITY;
    int32_t u_best = cmax;
    for (int m = warp + 1; m <= kMaxPieces; m += 32) {
        const int32_t U = (cmax + m - 1) / m;
        int32_t units = 0;
        float parts = 0.f, work = 0.f, longest = 0.f;
        for (int base = 0; base < n_pairs; base += 32) {
            const int q = base + lane;
            const int32_t c = q < n_pairs ? pairs[q].cost : 0;
            const int32_t k = q < n_pairs ? max((c + U - 1) / U, 1) : 0;
            int32_t incl = k;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            if (k > 0) {
                // the last multiple of N among the places of the pair's units
                const int32_t end = (units + incl) * a.Hkv, i = (end - 1) / p.ctas;
                if (i * p.ctas >= end - k * a.Hkv)
                    longest = fmaxf(longest, static_cast<float>(i + 1) * (static_cast<float>((c + k - 1) / k) + kUnitBlocks));
            }
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
        const float est = fmaxf(longest, heads * (work + kUnitBlocks * static_cast<float>(units)) / p.ctas);
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
    float e = best_est[lane];
    int32_t U = best_u[lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float oe = __shfl_xor_sync(0xffffffffu, e, d);
        const int32_t ou = __shfl_xor_sync(0xffffffffu, U, d);
        if (oe < e || (oe == e && ou > U)) {
            e = oe;
            U = ou;
        }
    }

    // unit and partial ranges
    int32_t ucarry = 0, pcarry = 0, scarry = 0;
    int32_t *splits = reinterpret_cast<int32_t *>(p.ws + p.lay.splits);
    for (int base = 0; base < n_pairs; base += kPlanT) {
        const int q = base + tid;
        int32_t k = 0, utotal, ptotal, stotal;
        if (q < n_pairs) k = max((pairs[q].cost + U - 1) / U, 1);
        const int32_t ku = scan_cta(k, sums, &utotal);
        const int32_t kp = scan_cta(k > 1 ? k : 0, sums, &ptotal);
        const int32_t ks = scan_cta(k > 1 ? 1 : 0, sums, &stotal);
        if (k > 1) splits[scarry + ks] = q;
        if (q < n_pairs) {
            pairs[q].unit0 = ucarry + ku;
            pairs[q].pieces = k;
            pairs[q].part0 = pcarry + kp;
        }
        ucarry += utotal;
        pcarry += ptotal;
        scarry += stotal;
    }
    // the sequences' unit ranges, from their first pairs'
    __syncthreads();
    for (int q = tid; q < n_pairs; q += kPlanT) {
        const int32_t next = pairs[q].seq_units, u0 = pairs[pairs[q].seq0].unit0;
        pairs[q].seq0 = u0;
        pairs[q].seq_units = (next < n_pairs ? pairs[next].unit0 : ucarry) - u0;
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
    if (blockIdx.x == 0) {
        plan_batch(p);
        return;
    }
    const ChunkArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t gwarp = (static_cast<int64_t>(blockIdx.x - 1) * kPlanT + threadIdx.x) / 32;
    const int64_t n_warps = static_cast<int64_t>(gridDim.x - 1) * (kPlanT / 32);

    // selection rows to bitmaps of key blocks, one warp a row
    if (a.tk != nullptr) {
        __shared__ uint32_t words[kPlanT / 32][kMaxNB / 32];
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
    const int bytes = (2 * p.a.B + 1) * static_cast<int>(sizeof(int32_t));
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(chunk_plan_kernel), bytes);
    if (e != cudaSuccess) return e;
    chunk_plan_kernel<<<device_sm_count(), kPlanT, bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace spd
