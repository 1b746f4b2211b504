// store.cuh -- device helpers of the cache stores: rounding to the kept type,
// and one head row normalised and rotated in fp32.
#pragma once

#include "f32x2.cuh"
#include "serve.cuh"
#include "spd_internal.cuh"

namespace spd {

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

// Head row h of token t of q (is_q) or k, normalised and rotated for position
// len - 1, by one warp: lane l gets dims l, l + 32, ... in x.  `row` is D floats
// of shared memory for the rotation partners.
constexpr int kPerLane = kMaxD / 32;
__device__ __forceinline__ void norm_rope_row(const StoreArgs &a, bool is_q, int64_t t, int h, int32_t len, float *row,
                                              float (&x)[kPerLane]) {
    const int lane = threadIdx.x & 31;
    const void *src = is_q ? a.q : a.k;
    const int64_t base = is_q ? t * a.q_s0 + h * a.q_s1 : t * a.k_s0 + h * a.k_s1;
    const int64_t ds = is_q ? a.q_s2 : a.k_s2;
    const void *w = is_q ? a.wq : a.wk;
    float ss = 0.f;
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
            if (d < a.D) x[c] *= inv * load_float(w, is_q ? a.wq_dt : a.wk_dt, d * (is_q ? a.wq_s0 : a.wk_s0));
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
        if (d >= a.Rd) continue;
        const int i = a.interleaved ? d >> 1 : (d < half ? d : d - half);  // angle of the pair
        const bool second = a.interleaved ? (d & 1) : d >= half;
        const float other = row[a.interleaved ? d ^ 1 : (second ? d - half : d + half)];
        const float co = cs[i * a.cs_s1], si = cs[(half + i) * a.cs_s1];
        x[c] = second ? fmaf(x[c], co, other * si) : fmaf(x[c], co, -(other * si));
    }
}

template <bool kBf16>
__device__ __forceinline__ uint64_t widen2(uint32_t u) {
    if (kBf16) return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
    return pair(f.x, f.y);
}

__device__ __forceinline__ uint64_t swapped(uint64_t x) {
    float lo, hi;
    unpair(x, lo, hi);
    return pair(hi, lo);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t round2(uint64_t x) {
    float lo, hi;
    unpair(x, lo, hi);
    if (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four neighbouring values, rounded and stored at p.
template <bool kBf16, bool kF8>
__device__ __forceinline__ void store4(void *p, uint64_t x0, uint64_t x1) {
    if (kF8) {
        float v[4];
        unpair(x0, v[0], v[1]);
        unpair(x1, v[2], v[3]);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
        *static_cast<uint32_t *>(p) = lo | (hi << 16);
    } else {
        *static_cast<uint2 *>(p) = make_uint2(round2<kBf16>(x0), round2<kBf16>(x1));
    }
}

}  // namespace spd
