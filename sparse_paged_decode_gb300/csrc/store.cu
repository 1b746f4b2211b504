// store.cu -- paged_norm_rope_store: per-head RMS norm and rotary positions
// of q and k, with K and V written into the paged caches.
//
// A head row of D elements is read once, normalised and rotated in fp32 and
// written once, rounded to the type it is kept in: the call moves its inputs
// and outputs and nothing else, so HBM bandwidth bounds it.  Measured, 64 + 8 +
// 8 rows of 128 dims a token into E4M3 caches: 61.7 us for 8192 tokens in a
// graph and 63.4 us called one by one (323 MB, 77 and 75 % of the measured copy
// bandwidth); 6.5 us for 466 tokens that the L2 holds, 8.9 us over buffers that
// it does not.
#include "spd_dispatch.h"
#include "store.cuh"

namespace spd {

namespace {

constexpr int kStoreWarps = 8;

// Any layout: one CTA per token, one warp per head row at a time, lane l
// holding dims l, l + 32, ...; the rotation partner comes through shared
// memory.
__global__ void __launch_bounds__(kStoreWarps * 32) store_generic_kernel(const StoreArgs a) {
    __shared__ float rows[kStoreWarps][kMaxD];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t len = a.tl[t * a.tl_s0];
    const int32_t slot = a.slots[t * a.slots_s0];
    const bool live = len >= 1 && len <= a.M;
    const bool stored = live && slot >= 0 && slot < a.n_slots;
    const int n_rows = a.Hq + a.Hkv * (a.v != nullptr ? 2 : 1);
    float *row = rows[warp];
    for (int r = warp; r < n_rows; r += kStoreWarps) {
        if (r >= a.Hq + a.Hkv) {  // a value row: copied
            if (!stored) continue;
            const int h = r - a.Hq - a.Hkv;
            for (int d = lane; d < a.D; d += 32) {
                const float x = load_float(a.v, a.in_dt, t * a.v_s0 + h * a.v_s1 + d * a.v_s2);
                store_as(a.vc, a.c_dt, slot * a.vc_s0 + h * a.vc_s1 + d * a.vc_s2, x * a.v_inv);
            }
            continue;
        }
        const bool is_q = r < a.Hq;
        const int h = is_q ? r : r - a.Hq;
        if (!live) {
            if (is_q)
                for (int d = lane; d < a.D; d += 32) store_as(a.qo, a.qo_dt, t * a.qo_s0 + h * a.qo_s1 + d * a.qo_s2, 0.f);
            continue;
        }
        if (!is_q && !stored) continue;
        float x[kPerLane];
        norm_rope_row(a, is_q, t, h, len, row, x);
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) {
            const int d = c * 32 + lane;
            if (d >= a.D) continue;
            if (is_q)
                store_as(a.qo, a.qo_dt, t * a.qo_s0 + h * a.qo_s1 + d * a.qo_s2, x[c]);
            else
                store_as(a.kc, a.c_dt, slot * a.kc_s0 + h * a.kc_s1 + d * a.kc_s2, x[c] * a.k_inv);
        }
    }
}

template <bool kBf16, bool kF8, int kLanes, int kMode>
__global__ void __launch_bounds__(kVecThreads, kVecCtas) store_vec_kernel(const StoreArgs a, int groups) {
    __shared__ __align__(16) float weights[2][8 * kLanes];
    load_weights<kLanes>(a, weights);
    store_rows<kBf16, kF8, kLanes, kMode, true>(a, weights, groups, blockIdx.x, gridDim.x);
}

template <bool kBf16, bool kF8, int kLanes>
void launch_vec(const StoreArgs &a, unsigned grid, int groups, cudaStream_t stream) {
    auto kernel = a.interleaved    ? store_vec_kernel<kBf16, kF8, kLanes, 2>
                  : a.Rd == a.D    ? store_vec_kernel<kBf16, kF8, kLanes, 0>
                                   : store_vec_kernel<kBf16, kF8, kLanes, 1>;
    kernel<<<grid, kVecThreads, 0, stream>>>(a, groups);
}

template <int kLanes>
void launch_vec(const StoreArgs &a, unsigned grid, int groups, cudaStream_t stream) {
    const bool bf16 = a.in_dt == SPD_BF16, f8 = a.c_dt == SPD_E4M3;
    if (bf16 && f8) launch_vec<true, true, kLanes>(a, grid, groups, stream);
    else if (bf16) launch_vec<true, false, kLanes>(a, grid, groups, stream);
    else if (f8) launch_vec<false, true, kLanes>(a, grid, groups, stream);
    else launch_vec<false, false, kLanes>(a, grid, groups, stream);
}

}  // namespace

cudaError_t launch_store_generic(const StoreArgs &a, cudaStream_t stream) {
    count_launches(1);
    store_generic_kernel<<<static_cast<unsigned>(a.T), kStoreWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

// 16-bit inputs of head dim 64, 128 or 256 with aligned contiguous rows, an
// output of their type, caches of their type or E4M3, and rotary dims in whole
// lanes.
bool store_vec_covers(const StoreArgs &a) {
    if (a.in_dt == SPD_F32 || a.qo_dt != a.in_dt || (a.c_dt != a.in_dt && a.c_dt != SPD_E4M3)) return false;
    if ((a.Hq - 1) * (a.q_s1 > 0 ? a.q_s1 : -a.q_s1) > INT32_MAX || (a.Hq - 1) * a.qo_s1 > INT32_MAX) return false;
    if (a.D != 64 && a.D != 128 && a.D != 256) return false;
    if (a.Rd % 8 != 0) return false;
    // base and row strides whole multiples of what a lane moves at a time
    auto rows_ok = [](const void *p, int bytes, int es, int64_t s0, int64_t s1, int64_t s2) {
        return s2 == 1 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s0 * es) % bytes == 0 && (s1 * es) % bytes == 0;
    };
    const int ces = a.c_dt == SPD_E4M3 ? 1 : 2;
    if (!rows_ok(a.q, 8, 2, a.q_s0, a.q_s1, a.q_s2) || !rows_ok(a.k, 8, 2, a.k_s0, a.k_s1, a.k_s2) ||
        !rows_ok(a.qo, 8, 2, a.qo_s0, a.qo_s1, a.qo_s2) || !rows_ok(a.kc, 4 * ces, ces, a.kc_s0, a.kc_s1, a.kc_s2) ||
        !rows_ok(a.cs, 16, 4, a.cs_s0, 0, a.cs_s1))
        return false;
    if (a.v != nullptr &&
        (!rows_ok(a.v, 8, 2, a.v_s0, a.v_s1, a.v_s2) || !rows_ok(a.vc, 4 * ces, ces, a.vc_s0, a.vc_s1, a.vc_s2)))
        return false;
    return true;
}

// As many row groups to a token as its rows can use.
int store_row_groups(const StoreArgs &a, int n_kv) {
    const int lanes = a.D / 8, n_q = (a.Hq + kQRows - 1) / kQRows, most = n_kv > n_q ? n_kv : n_q;
    int groups = 1;
    while (groups < most && groups < kVecThreads / lanes) groups *= 2;
    return groups;
}

// Anything that store_vec_covers does not: *used stays false.
cudaError_t launch_store_vec(const StoreArgs &a, cudaStream_t stream, bool *used) {
    *used = false;
    if (!store_vec_covers(a)) return cudaSuccess;
    const int lanes = a.D / 8, n_kv = a.Hkv * (a.v != nullptr ? 2 : 1);
    const int groups = store_row_groups(a, n_kv);
    const int tokens = kVecThreads / lanes / groups;
    const int64_t want = (static_cast<int64_t>(a.T) + tokens - 1) / tokens, room = static_cast<int64_t>(device_sm_count()) * kVecCtas;
    const unsigned grid = static_cast<unsigned>(want < room ? want : room);
    if (lanes == 8) launch_vec<8>(a, grid, groups, stream);
    else if (lanes == 16) launch_vec<16>(a, grid, groups, stream);
    else launch_vec<32>(a, grid, groups, stream);
    count_launches(1);
    *used = true;
    return cudaGetLastError();
}

}  // namespace spd
