// block_scale.cuh -- how the tensor-core attention kernels take the scales of
// block-scaled E4M3 caches (one K and one V scale a page and kv head).
//
// With ks and vs the scales of a key's page, z its logit in log2 units and m
// the row's running offset,
//   z  = ks (q . k) c,   w = 2^(z + log2 vs - m),   O += w v,   l += w / vs
// so O / l = sum 2^z vs v / sum 2^z: the V scale enters through the exponent.
// The offset is a maximum of z + log2 vs, so the weights that are rounded to
// 16 bits are relative to the largest product of weight and scale, whatever the
// scales' range; no scaled copy of V is made, and partial sums of a row join as
// without scales.  (A scale in the widened f16 values instead would leave the
// range of f16 for scales 2^8 apart.)
//
// The sum has a wider range than the weights.  A page's scale may be 2^-128 of
// another's, and ex2 gives 0 below 2^-126, so w may be lost where its key's softmax
// weight is not.  Pages of scales below 2^kLowScale therefore add 2^(z - m) itself, an
// exponential more a key (the kernel of single rows, which HBM bounds, adds it for
// every page); any other page lies within 2^96 of all, and a w that is 0 there belongs
// to a key of less than 2^-30 of the softmax weight of the key that the offset comes
// from.  z - m is at most 64 and the raise's headroom, and the sum at least 2^-64, so
// it is brought to a new offset in two steps (`rescale`).
//
// The loading thread copies a page's two scales beside its keys, with cp.async
// and an arrival on the same barrier: a ring of kScaleRing pages, which no
// loader runs ahead of (each kernel says why).
#pragma once

#include "spd_internal.cuh"
#include "tc_ptx.cuh"

namespace spd {

constexpr float kLowScale = -32.f;  // log2

struct BlockScale {
    float k, lg_v, inv_v;  // the K scale, log2 of the V scale, its reciprocal: 0 for a low one
};

// The sum adds its keys' 2^(z - m) for this page, not w / vs.
__device__ __forceinline__ bool low_scale(const BlockScale &s) { return s.inv_v == 0.f; }

// A sum times 2^by, by <= 0 of any size (-inf: 0).  Returns 2^by.
__device__ __forceinline__ float rescale(float &l, float by) {
    const float root = tc::ex2(0.5f * by);
    l = l * root * root;
    return root * root;
}

__device__ __forceinline__ BlockScale block_scale(float2 kv) {
    BlockScale s;
    const float v = clip_scale(kv.y);
    const uint32_t bits = __float_as_uint(v);
    s.k = clip_scale(kv.x);
    // exponent and significand apart: exact for powers of two.  Else off by the
    // logarithm's 2^-22 and the rounding of the sum, up to 2^-19 for scales from 2^32
    // on (or below 2^-32), which a weight takes over as 0.7 times that of itself
    s.lg_v = static_cast<float>(static_cast<int>(bits >> 23) - 127) +
             __log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
    // of the very factor that the exponent carries, and one instruction where a
    // division takes ten, for every thread and page (prefill dense 518 -> 507 us)
    s.inv_v = s.lg_v < kLowScale ? 0.f : tc::ex2(-s.lg_v);
    return s;
}

// The two scales of a page and head on their way to `dst`, arriving on `bar`.
__device__ __forceinline__ void load_block_scale(float2 *dst, const PageScales &sc, int64_t page, int h, uint64_t *bar) {
    tc::cp_async4(&dst->x, sc.k + page * sc.k_s0 + h * sc.k_s1);
    tc::cp_async4(&dst->y, sc.v + page * sc.v_s0 + h * sc.v_s1);
    tc::cp_async_arrive(bar);
}

}  // namespace spd
