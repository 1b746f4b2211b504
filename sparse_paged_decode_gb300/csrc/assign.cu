// assign.cu -- paged_assign_slots: the page table grown from a free list and
// every token's row, length and slot, from the requests' lengths alone.
//
// Everything follows from two prefix sums over the requests: of the new
// tokens (clipped to the T token rows), and then of the blocks each request
// grows by and of its query blocks.  The sums are a few thousand integers at
// most, so every CTA makes them for itself in shared memory instead of
// waiting for another kernel: the call is one launch with no workspace.  CTA
// c then fills its share of the token rows and of the grown table cells, and
// CTA 0 the per-request outputs.  A token on a grown block takes its page
// straight from the free list (the same entry that the table cell gets), so
// no token waits for the table to be written.
//
// What bounds it is latency: a launch and three dependent reads (lengths, the
// page of a token, the write).  Measured in a graph: 4.6 us for 466 tokens of
// 64 requests, 6.2 us for 65536 tokens of 1024 (0.8 MB, 0.1 us of HBM time; four
// tokens to a thread, on a quarter of the CTAs, took 8.8 us); 6.2 and 8.2 us
// called one by one.
#include "serve.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"

namespace spd {

namespace {

constexpr int kAssignThreads = 512;
constexpr int kTokensPerCta = 512;

__device__ __forceinline__ int32_t clip0(int64_t x, int64_t hi) {
    return static_cast<int32_t>(x < 0 ? 0 : (x > hi ? hi : x));
}

// Exclusive prefix sum over the CTA's threads, and the total; sums saturate
// at `cap` (saturated addition of non-negative numbers is associative).
__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t cap, int32_t *warp_sums, int32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = min(incl + y, cap);
    }
    int32_t excl = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) excl = 0;
    __syncthreads();  // an earlier scan's readers of warp_sums are done
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    constexpr int kWarps = kAssignThreads / 32;
    int32_t w = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w = min(w + y, cap);
    }
    const int32_t before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
    return min(before + excl, cap);
}

// Largest b in [0, n) with off[b] <= x (off[0] = 0, nondecreasing, off[n] > x).
__device__ __forceinline__ int find(const int32_t *off, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kAssignThreads) assign_kernel(const AssignArgs a) {
    extern __shared__ int32_t sh[];
    __shared__ int32_t warp_sums[kAssignThreads / 32];
    int32_t *cu = sh;                // [B + 1] token offsets
    int32_t *go = sh + a.B + 1;      // [B + 1] grown-block offsets
    const int tid = threadIdx.x;
    const int64_t cap = static_cast<int64_t>(a.NB) * kBlock;
    const int per = (a.B + kAssignThreads - 1) / kAssignThreads;  // requests of a thread
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    const int32_t count = clip0(a.free_count[0], a.F);

    // token offsets, clipped to T
    int32_t sum = 0, total = 0;
    for (int b = b0; b < b1; ++b) sum = min(sum + clip0(a.nw[b * a.nw_s0], a.T), a.T);
    int32_t at = block_scan(sum, a.T, warp_sums, &total);
    for (int b = b0; b < b1; ++b) {
        cu[b] = at;
        at = min(at + clip0(a.nw[b * a.nw_s0], a.T), a.T);
    }
    if (tid == 0) cu[a.B] = total;
    const int32_t n_tokens = total;
    __syncthreads();

    // blocks each request grows by, and its query blocks
    auto grown = [&](int b) -> int32_t {
        const int32_t n = cu[b + 1] - cu[b], r = a.sid[b * a.sid_s0];
        if (r < 0 || r >= a.R) return 0;
        const int64_t p = max(a.pre[b * a.pre_s0], 0);
        return static_cast<int32_t>((min(p + n, cap) + kBlock - 1) / kBlock - (min(p, cap) + kBlock - 1) / kBlock);
    };
    sum = 0;
    int32_t qsum = 0;
    for (int b = b0; b < b1; ++b) {
        sum += grown(b);
        const int32_t n = cu[b + 1] - cu[b];
        qsum += n / a.bsq + (n % a.bsq != 0);
    }
    int32_t qtotal = 0;
    at = block_scan(sum, INT32_MAX / 2, warp_sums, &total);
    int32_t qat = block_scan(qsum, INT32_MAX / 2, warp_sums, &qtotal);
    const bool first_cta = blockIdx.x == 0;
    for (int b = b0; b < b1; ++b) {
        go[b] = at;
        at += grown(b);
        if (first_cta) {
            const int32_t n = cu[b + 1] - cu[b];
            a.cu[b * a.cu_s0] = cu[b];
            a.cub[b * a.cub_s0] = qat;
            qat += n / a.bsq + (n % a.bsq != 0);
            const int64_t whole = static_cast<int64_t>(max(a.pre[b * a.pre_s0], 0)) + n;
            a.sl[b * a.sl_s0] = static_cast<int32_t>(min(whole, static_cast<int64_t>(INT32_MAX)));
        }
    }
    if (tid == 0) {
        go[a.B] = total;
        if (first_cta) {
            a.cu[a.B * a.cu_s0] = n_tokens;
            a.cub[a.B * a.cub_s0] = qtotal;
            a.left[0] = max(count - total, 0);
        }
    }
    const int32_t n_grown = total;
    __syncthreads();

    // grown table cells: the i-th takes the i-th free page from the end
    const int stride = gridDim.x * kAssignThreads;
    for (int i = blockIdx.x * kAssignThreads + tid; i < n_grown; i += stride) {
        const int b = find(go, a.B, i);
        const int64_t p = max(a.pre[b * a.pre_s0], 0);
        const int64_t blk = (p + kBlock - 1) / kBlock + (i - go[b]);
        const int32_t page = i < count ? a.free_pages[static_cast<int64_t>(count - 1 - i) * a.fp_s0] : -1;
        a.bt[a.sid[b * a.sid_s0] * a.bt_s0 + blk * a.bt_s1] = page;
    }

    // token rows
    for (int t = blockIdx.x * kAssignThreads + tid; t < a.T; t += stride) {
        int32_t req = -1, len = 0, slot = -1;
        if (t < n_tokens) {
            const int b = find(cu, a.B, t);
            req = a.sid[b * a.sid_s0];
            const int64_t p = max(a.pre[b * a.pre_s0], 0), pos = p + (t - cu[b]);
            len = static_cast<int32_t>(min(pos + 1, static_cast<int64_t>(INT32_MAX)));
            if (req >= 0 && req < a.R && pos < cap) {
                const int64_t blk = pos / kBlock, first = (p + kBlock - 1) / kBlock;
                int32_t page;
                if (blk >= first) {
                    const int64_t i = go[b] + (blk - first);
                    page = i < count ? a.free_pages[(count - 1 - i) * a.fp_s0] : -1;
                } else {
                    page = a.bt[req * a.bt_s0 + blk * a.bt_s1];
                }
                if (page >= 0 && page < a.n_pages) slot = page * kBlock + static_cast<int32_t>(pos % kBlock);
            }
        }
        a.req[t * a.req_s0] = req;
        a.tl[t * a.tl_s0] = len;
        a.slots[t * a.slots_s0] = slot;
    }
}

}  // namespace

cudaError_t launch_assign(const AssignArgs &a, cudaStream_t stream) {
    const int bytes = 2 * (a.B + 1) * static_cast<int>(sizeof(int32_t));
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(assign_kernel), bytes);
    if (e != cudaSuccess) return e;
    const int want = (a.T + kTokensPerCta - 1) / kTokensPerCta;
    const int grid = want < 1 ? 1 : (want > device_sm_count() ? device_sm_count() : want);
    count_launches(1);
    assign_kernel<<<grid, kAssignThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace spd
