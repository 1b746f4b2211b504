// store.cu -- paged_norm_rope_store: per-head RMS norm and rotary positions
// of q and k, with K and V written into the paged caches.
//
// A head row of D elements is read once, normalised and rotated in fp32 and
// written once, rounded to the type it is kept in: the call moves its inputs
// and outputs and nothing else, so HBM bandwidth bounds it.
#include "serve.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"

namespace spd {

namespace {

constexpr int kStoreWarps = 8;
constexpr int kPerLane = kMaxD / 32;

// x rounded to the type dt and stored at element `off` of base.  E4M3 rounds
// to nearest even, saturates at +-448 and keeps NaN.
__device__ __forceinline__ void store_as(void *base, int dt, int64_t off, float x) {
    if (dt == SPD_F32) {
        static_cast<float *>(base)[off] = x;
    } else if (dt == SPD_BF16) {
        static_cast<__nv_bfloat16 *>(base)[off] = __float2bfloat16_rn(x);
    } else if (dt == SPD_F16) {
        static_cast<__half *>(base)[off] = __float2half_rn(x);
    } else {
        static_cast<uint8_t *>(base)[off] = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    }
}

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
        const void *src = is_q ? a.q : a.k;
        const int64_t base = is_q ? t * a.q_s0 + h * a.q_s1 : t * a.k_s0 + h * a.k_s1;
        const int64_t ds = is_q ? a.q_s2 : a.k_s2;
        const void *w = is_q ? a.wq : a.wk;
        float x[kPerLane], ss = 0.f;
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) {
            const int d = c * 32 + lane;
            x[c] = d < a.D ? load_float(src, a.in_dt, base + d * ds) : 0.f;
            ss = fmaf(x[c], x[c], ss);
        }
        if (w != nullptr) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float inv = rsqrtf(ss / a.D + a.eps);
#pragma unroll
            for (int c = 0; c < kPerLane; ++c) {
                const int d = c * 32 + lane;
                if (d < a.D)
                    x[c] *= inv * load_float(w, is_q ? a.wq_dt : a.wk_dt, d * (is_q ? a.wq_s0 : a.wk_s0));
            }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kPerLane; ++c)
            if (c * 32 + lane < a.D) row[c * 32 + lane] = x[c];
        __syncwarp();
        const float *cs = a.cs + static_cast<int64_t>(len - 1) * a.cs_s0;
        const int half = a.Rd / 2;
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) {
            const int d = c * 32 + lane;
            if (d >= a.D) continue;
            float y = x[c];
            if (d < a.Rd) {
                const int i = a.interleaved ? d >> 1 : (d < half ? d : d - half);  // angle of the pair
                const bool second = a.interleaved ? (d & 1) : d >= half;
                const float other = row[a.interleaved ? d ^ 1 : (second ? d - half : d + half)];
                const float co = cs[i * a.cs_s1], si = cs[(half + i) * a.cs_s1];
                y = second ? fmaf(y, co, other * si) : fmaf(y, co, -(other * si));
            }
            if (is_q)
                store_as(a.qo, a.qo_dt, t * a.qo_s0 + h * a.qo_s1 + d * a.qo_s2, y);
            else
                store_as(a.kc, a.c_dt, slot * a.kc_s0 + h * a.kc_s1 + d * a.kc_s2, y * a.k_inv);
        }
    }
}

}  // namespace

cudaError_t launch_store_generic(const StoreArgs &a, cudaStream_t stream) {
    count_launches(1);
    store_generic_kernel<<<static_cast<unsigned>(a.T), kStoreWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace spd
