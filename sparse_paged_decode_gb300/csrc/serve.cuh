// serve.cuh -- argument blocks and launchers of the serving-step calls around
// the paged caches (paged_assign_slots, paged_norm_rope_store and the prefill
// attention calls).  Internal to the library; nothing here is part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "spd_internal.cuh"

namespace spd {

constexpr int kMaxSeqs = 8192;  // requests of one call

struct AssignArgs {
    const int32_t *nw, *pre, *sid;  // [B] new tokens, cached tokens, page-table row
    int64_t nw_s0, pre_s0, sid_s0;
    const int32_t *free_pages;      // [F]
    int64_t fp_s0;
    const int32_t *free_count;      // [1]
    int32_t *bt;                    // [R, NB] in/out
    int64_t bt_s0, bt_s1;
    int32_t *cu, *cub, *sl;         // [B+1], [B+1], [B]
    int64_t cu_s0, cub_s0, sl_s0;
    int32_t *req, *tl, *slots;      // [T]
    int64_t req_s0, tl_s0, slots_s0;
    int32_t *left;                  // [1]
    int32_t B, F, R, NB, T, n_pages, bsq;
};

cudaError_t launch_assign(const AssignArgs &a, cudaStream_t stream);

struct StoreArgs {
    const void *q, *k, *v;          // [T, Hq, D], [T, Hkv, D], [T, Hkv, D] or null
    int64_t q_s0, q_s1, q_s2, k_s0, k_s1, k_s2, v_s0, v_s1, v_s2;
    const void *wq, *wk;            // [D] or null
    int64_t wq_s0, wk_s0;
    const float *cs;                // [M, Rd]
    int64_t cs_s0, cs_s1;
    const int32_t *tl, *slots;      // [T]
    int64_t tl_s0, slots_s0;
    void *qo;                       // [T, Hq, D]
    int64_t qo_s0, qo_s1, qo_s2;
    void *kc, *vc;                  // [P*128, Hkv, D]
    int64_t kc_s0, kc_s1, kc_s2, vc_s0, vc_s1, vc_s2;
    int64_t n_slots;                // P*128
    int32_t in_dt, wq_dt, wk_dt, qo_dt, c_dt;
    int32_t T, Hq, Hkv, D, Rd, M;
    int32_t interleaved;
    float eps, k_inv, v_inv;        // reciprocal scales
    float *ks, *vs;                 // [P, Hkv] scales of block-scaled caches, or null
    int64_t ks_s0, ks_s1, vs_s0, vs_s1;
};

cudaError_t launch_store_generic(const StoreArgs &a, cudaStream_t stream);
cudaError_t launch_store_vec(const StoreArgs &a, cudaStream_t stream, bool *used);
bool store_vec_covers(const StoreArgs &a);       // shapes and layouts of the vector kernels
int store_row_groups(const StoreArgs &a, int n_kv);
cudaError_t dispatch_store(const StoreArgs &a, cudaStream_t stream);

cudaError_t launch_store_block_generic(const StoreArgs &a, cudaStream_t stream);
cudaError_t launch_store_block_vec(const StoreArgs &a, cudaStream_t stream, bool *used);
cudaError_t dispatch_store_block(const StoreArgs &a, cudaStream_t stream);

struct ChunkArgs {
    const void *q;                  // [total_q, Hq, D]
    int64_t q_s0, q_s1, q_s2;
    const uint8_t *k, *v;           // [P*128, Hkv, D], innermost stride 1
    int64_t k_s0, k_s1, v_s0, v_s1;
    const int32_t *bt;              // [R, NB]
    int64_t bt_s0, bt_s1;
    const int32_t *sid, *cu, *sl, *pre;  // [B], [B+1], [B], [B]
    int64_t sid_s0, cu_s0, sl_s0, pre_s0;
    const int32_t *tk;              // [Hkv, n_rows, K] or null (every block)
    int64_t tk_s0, tk_s1, tk_s2;
    const int32_t *cub;             // [B+1] or null
    int64_t cub_s0;
    void *out;                      // [total_q, Hq, D] bf16
    int64_t o_s0, o_s1, o_s2;
    int32_t q_dt, kv_dt;
    int32_t total_q, Hq, Hkv, D, B, R, NB, n_rows, K, bsq;
    int64_t P;
    float sm_scale, k_scale, v_scale;  // the last two 1 for block-scaled caches
    PageScales sc;
};

cudaError_t launch_chunk_generic(const ChunkArgs &a, cudaStream_t stream);
cudaError_t dispatch_chunk(const ChunkArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t chunk_workspace_bytes(int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t NB,
                             int64_t n_rows);

// Kernel policy of the prefill attention calls (5) and the store (6); -1 for
// another stage.
int set_serve_policy(int stage, int policy);

#ifdef __CUDACC__
// Sequence that owns query token t under the offsets cu [B+1] (stride s): the
// last b in [0, B) with cu[b] <= t, or -1 when there is none or t is at or
// past cu[b+1].
__device__ __forceinline__ int owning_sequence(const int32_t *cu, int64_t s, int B, int64_t t) {
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi] once lo is known to hold
    if (B <= 0 || cu[0] > t) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid * s] <= t) lo = mid; else hi = mid;
    }
    return t < cu[(lo + 1) * s] ? lo : -1;
}

// Keys token i of sequence b may read: min(prefix + i + 1, seq_len, NB * 128),
// 0 when the sequence's page-table row is outside the table.
__device__ __forceinline__ int32_t chunk_limit(const ChunkArgs &a, int b, int64_t i) {
    const int32_t r = a.sid[b * a.sid_s0];
    if (r < 0 || r >= a.R) return 0;
    int64_t L = static_cast<int64_t>(a.pre[b * a.pre_s0]) + i + 1;
    const int64_t sl = a.sl[b * a.sl_s0], cap = static_cast<int64_t>(a.NB) * 128;
    if (L > sl) L = sl;
    if (L > cap) L = cap;
    return L < 0 ? 0 : static_cast<int32_t>(L);
}
#endif

}  // namespace spd
