// store_block.cu -- paged_norm_rope_store_block_scaled: per-head RMS norm and
// rotary positions of q and k, with K and V appended to E4M3 pages that have
// one scale for each page and kv head.
//
// The stored rows of a page are a run: neighbouring rows of the batch whose
// slots rise by one.  For a head of a run whose first slot has offset f in its
// page, with y the rows to be kept (K normalised and rotated, V as it is),
//   need  = the smallest 2^e, e in [-64, 64], with max |y| <= 448 * 2^e
//   old   = the page's scale, none where f = 0: the page is begun anew
//   scale = old where old >= need, else need
//   codes of offsets 0 .. f-1 are multiplied by old / scale, those of the run
//   are y / scale, each rounded once.
// Powers of two: E4M3 is a floating format, so a scale between them keeps no
// more bits, and a page that grows moves its codes by whole exponents, which
// rounds only those that become subnormal.  The maximum is taken over finite
// elements (an infinity saturates, a NaN stays one) and does not depend on an
// order.
#include "spd_dispatch.h"
#include "store.cuh"

namespace spd {

namespace {

constexpr int kWarps = 8;
constexpr int kLeastExp = -64, kMostExp = 64;  // of the scales that are written

// The smallest 2^e with `top` <= 448 * 2^e = 1.75 * 2^(e + 8): the exponent of
// top, less 8, plus one where its significand is above 1.75.
__device__ __forceinline__ float scale_of(float top) {
    const int e = static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8;
    return __uint_as_float(static_cast<uint32_t>(127 + max(kLeastExp, min(kMostExp, e))) << 23);
}

// |x| where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
    const float m = fabsf(x);
    return m < INFINITY ? m : 0.f;
}

// The scale of a page and head whose new rows reach `top`, and what its held
// codes (offsets below f) are multiplied by: 1 where they stay as they are.
__device__ __forceinline__ float page_scale(float top, const float *at, int f, float &ratio) {
    const float need = scale_of(top);
    const float old = f > 0 ? *at : 0.f;
    ratio = 1.f;
    if (!(old > 0.f && old < INFINITY)) return need;  // no scale: nothing that it could have scaled
    if (old >= need) return old;
    ratio = old / need;
    return need;
}

__device__ __forceinline__ uint8_t rescaled(uint8_t code, float ratio) {
    return __nv_cvt_float_to_fp8(e4m3_to_float(code) * ratio, __NV_SATFINITE, __NV_E4M3);
}

struct Row {
    int32_t len, slot;
    bool live, stored;
};

__device__ __forceinline__ Row row_of(const StoreArgs &a, int64_t t) {
    Row r;
    r.len = a.tl[t * a.tl_s0];
    r.slot = a.slots[t * a.slots_s0];
    r.live = r.len >= 1 && r.len <= a.M;
    r.stored = r.live && r.slot >= 0 && r.slot < a.n_slots;
    return r;
}

// Any layout: one CTA per batch row.  It writes the row's queries, and where
// the row begins a run it appends the whole run, one warp per K or V head: once
// over the run's rows for the maximum, once more to store them.
__global__ void __launch_bounds__(kWarps * 32) store_block_generic_kernel(const StoreArgs a) {
    __shared__ float rows[kWarps][kMaxD];
    __shared__ int run;
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Row r = row_of(a, t);
    float *row = rows[warp];
    float x[kPerLane];
    for (int h = warp; h < a.Hq; h += kWarps) {
        if (r.live) norm_rope_row(a, true, t, h, r.len, row, x);
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) {
            const int d = c * 32 + lane;
            if (d < a.D) store_as(a.qo, a.qo_dt, t * a.qo_s0 + h * a.qo_s1 + d * a.qo_s2, r.live ? x[c] : 0.f);
        }
    }
    if (!r.stored) return;
    const int f = r.slot % kBlock;
    const int64_t page = r.slot / kBlock;
    if (f > 0 && t > 0) {
        const Row before = row_of(a, t - 1);
        if (before.stored && before.slot == r.slot - 1) return;  // inside a run
    }
    if (threadIdx.x == 0) run = kBlock - f;
    __syncthreads();
    if (threadIdx.x < kBlock - f) {
        const int i = threadIdx.x;
        const bool in = t + i < a.T;
        const Row next = in ? row_of(a, t + i) : Row{0, 0, false, false};
        if (!next.stored || next.slot != r.slot + i) atomicMin(&run, i);
    }
    __syncthreads();
    const int n = run;
    for (int u = warp; u < 2 * a.Hkv; u += kWarps) {
        const bool is_k = u < a.Hkv;
        const int h = is_k ? u : u - a.Hkv;
        auto load = [&](int i) {
            if (is_k) {
                norm_rope_row(a, false, t + i, h, a.tl[(t + i) * a.tl_s0], row, x);
            } else {
#pragma unroll
                for (int c = 0; c < kPerLane; ++c) {
                    const int d = c * 32 + lane;
                    x[c] = d < a.D ? load_float(a.v, a.in_dt, (t + i) * a.v_s0 + h * a.v_s1 + d * a.v_s2) : 0.f;
                }
            }
        };
        float top = 0.f;
        for (int i = 0; i < n; ++i) {
            load(i);
#pragma unroll
            for (int c = 0; c < kPerLane; ++c) top = fmaxf(top, finite_abs(x[c]));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        float *at = is_k ? a.ks + page * a.ks_s0 + h * a.ks_s1 : a.vs + page * a.vs_s0 + h * a.vs_s1;
        float ratio;
        const float scale = page_scale(top, at, f, ratio), inv = 1.f / scale;
        __syncwarp();
        if (lane == 0) *at = scale;
        uint8_t *cache = static_cast<uint8_t *>(is_k ? a.kc : a.vc);
        const int64_t s0 = is_k ? a.kc_s0 : a.vc_s0, s1 = is_k ? a.kc_s1 : a.vc_s1, s2 = is_k ? a.kc_s2 : a.vc_s2;
        if (ratio != 1.f)
            for (int i = 0; i < f; ++i)
                for (int d = lane; d < a.D; d += 32) {
                    uint8_t *code = cache + (page * kBlock + i) * s0 + h * s1 + d * s2;
                    *code = rescaled(*code, ratio);
                }
        for (int i = 0; i < n; ++i) {
            load(i);
#pragma unroll
            for (int c = 0; c < kPerLane; ++c) {
                const int d = c * 32 + lane;
                if (d < a.D) store_as(cache, SPD_E4M3, (r.slot + i) * s0 + h * s1 + d * s2, x[c] * inv);
            }
        }
    }
}

}  // namespace

cudaError_t launch_store_block_generic(const StoreArgs &a, cudaStream_t stream) {
    count_launches(1);
    store_block_generic_kernel<<<static_cast<unsigned>(a.T), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace spd
