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
#include "f32x2.cuh"
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

// 16-bit rows of D = 8 * kLanes dims: kLanes lanes hold a head row, eight dims
// to a lane, as two runs of four: the runs that rotate with one another where
// the partners lie half the rotary dims apart, neighbouring runs elsewhere.  So
// the rotation needs no exchange between lanes, and the norm's sum is the only
// one.  With weights g and the row's factor f = 1 / sqrt(mean(x^2) + eps),
//   y_a = f (x_a (g_a cos) - x_b (g_b sin)),  y_b = f (x_b (g_b cos) + x_a (g_a sin)):
// the bracketed products are a token's, not a row's, and made once for all of
// its query rows.  A lane takes the same dims of every row, kQRows query rows
// and one K or V row at a time, loaded before the first is used and without
// waiting for the token's length.  Instructions, then HBM, bound the kernel:
// with the partner in another lane and the weights applied row by row it took
// 180 instructions a warp and row pair, and 74 us for the 8192 tokens.
constexpr int kVecThreads = 256;
constexpr int kVecCtas = 3;  // on an SM
constexpr int kQRows = 4;

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

// kF8: E4M3 caches, else caches of the inputs' type.  kMode 0: partners half
// the rotary dims apart, every dim turns; 1: the same, some dims do not turn;
// 2: neighbouring partners.  Row offsets within a token fit 32 bits.
template <bool kBf16, bool kF8, int kLanes, int kMode>
__global__ void __launch_bounds__(kVecThreads, kVecCtas) store_vec_kernel(const StoreArgs a, int groups) {
    __shared__ __align__(16) float weights[2][8 * kLanes];
    for (int i = threadIdx.x; i < 16 * kLanes; i += kVecThreads) {
        const int d = i % (8 * kLanes);
        const bool of_q = i < 8 * kLanes;
        const void *wt = of_q ? a.wq : a.wk;
        weights[of_q ? 0 : 1][d] =
            wt == nullptr ? 1.f : load_float(wt, of_q ? a.wq_dt : a.wk_dt, d * (of_q ? a.wq_s0 : a.wk_s0));
    }
    __syncthreads();

    // `groups` row groups share a token; the CTA's others take its next tokens
    const int gid = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, row0 = gid % groups;
    const int tokens = kVecThreads / kLanes / groups;
    const int half = a.Rd / 2, n_kv = a.Hkv * (a.v != nullptr ? 2 : 1);
    constexpr int ces = kF8 ? 1 : 2;
    const bool norm_q = a.wq != nullptr, norm_k = a.wk != nullptr;
    const int q_s1 = static_cast<int>(a.q_s1), qo_s1 = static_cast<int>(a.qo_s1);
    // this lane's runs of four dims
    const bool turns = kMode == 0 || (kMode == 1 ? 4 * lane < half : 8 * lane < a.Rd);
    const int da = kMode == 2 ? 8 * lane : (turns ? 4 * lane : a.Rd + 8 * (lane - half / 4));
    const int db = kMode == 2 || !turns ? da + 4 : half + 4 * lane;

    // what a row's four pairs are multiplied by, from the weights g and the
    // angles' cosines and sines: y = x * own + partner * cross
    auto factors = [&](const float *g, float4 c, float4 s, uint64_t *own, uint64_t *cross) {
        const float4 ga = *reinterpret_cast<const float4 *>(g + da), gb = *reinterpret_cast<const float4 *>(g + db);
        if (kMode == 2) {  // pairs (0, 1), (2, 3), ..: one angle each, partner in the same pair
            own[0] = pair(ga.x * c.x, ga.y * c.x); cross[0] = pair(-ga.y * s.x, ga.x * s.x);
            own[1] = pair(ga.z * c.y, ga.w * c.y); cross[1] = pair(-ga.w * s.y, ga.z * s.y);
            own[2] = pair(gb.x * c.z, gb.y * c.z); cross[2] = pair(-gb.y * s.z, gb.x * s.z);
            own[3] = pair(gb.z * c.w, gb.w * c.w); cross[3] = pair(-gb.w * s.w, gb.z * s.w);
        } else {  // first run against second, four angles
            own[0] = pair(ga.x * c.x, ga.y * c.y); cross[0] = pair(-gb.x * s.x, -gb.y * s.y);
            own[1] = pair(ga.z * c.z, ga.w * c.w); cross[1] = pair(-gb.z * s.z, -gb.w * s.w);
            own[2] = pair(gb.x * c.x, gb.y * c.y); cross[2] = pair(ga.x * s.x, ga.y * s.y);
            own[3] = pair(gb.z * c.z, gb.w * c.w); cross[3] = pair(ga.z * s.z, ga.w * s.w);
        }
    };

    // A row's sum of squares is exchanged by shuffles that name the whole warp,
    // so a warp's lanes take the same branches and turns: its row groups may
    // belong to different tokens, and have different numbers of rows (three
    // heads on groups of two, say), so what all of them do goes by the first of
    // them, and a group without a row of its own works on zeros.  (Naming a
    // row's own lanes instead took 6 % more: 65.2 us for the 8192 tokens, not
    // 61.3.)
    const int first = row0 & ~(32 / kLanes - 1), behind = row0 - first;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * tokens;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * tokens; base < a.T; base += stride) {
        const int64_t t = base + gid / groups;
        const bool in = t < a.T;
        const int32_t len = in ? a.tl[t * a.tl_s0] : 0;
        const int32_t slot = in ? a.slots[t * a.slots_s0] : -1;
        const bool live = len >= 1 && len <= a.M;
        const bool stored = live && slot >= 0 && slot < a.n_slots;
        const uint16_t *qa = static_cast<const uint16_t *>(a.q) + t * a.q_s0 + da;
        uint16_t *oa = static_cast<uint16_t *>(a.qo) + t * a.qo_s0 + da;
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
        uint64_t own[4], cross[4];

        // y of one row; the row's factor is 1 without a norm
        auto turn = [&](const uint64_t *x, bool norm, uint64_t *y) {
            float f = 1.f;
            if (norm) {
                const uint64_t sq = fma2(x[3], x[3], fma2(x[2], x[2], fma2(x[1], x[1], mul2(x[0], x[0]))));
                float lo, hi;
                unpair(sq, lo, hi);
                float ss = lo + hi;
#pragma unroll
                for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                f = rsqrtf(fmaf(ss, 1.f / (8 * kLanes), a.eps));
            }
            const uint64_t f2 = pair(f, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t partner = kMode == 2 ? swapped(x[e]) : x[e ^ 2];
                y[e] = mul2(x[e], own[e]);
                // dims that do not turn take nothing: 0 times what is not finite is not 0
                if (kMode == 0 || turns) y[e] = fma2(partner, cross[e], y[e]);
                y[e] = mul2(y[e], f2);
            }
        };

        for (int wq = first, wk = first; wq < a.Hq || wk < n_kv; wq += kQRows * groups, wk += groups) {
            const int rq = wq + behind, rk = wk + behind;
            uint2 wa[kQRows + 1], wb[kQRows + 1];
#pragma unroll
            for (int i = 0; i < kQRows; ++i) {
                const int r = rq + i * groups;
                wa[i] = wb[i] = make_uint2(0, 0);
                if (in && r < a.Hq) {
                    const uint16_t *src = qa + r * q_s1;
                    wa[i] = *reinterpret_cast<const uint2 *>(src);
                    wb[i] = *reinterpret_cast<const uint2 *>(src + (db - da));
                }
            }
            const bool is_k = rk < a.Hkv;
            const int hk = is_k ? rk : rk - a.Hkv;
            wa[kQRows] = wb[kQRows] = make_uint2(0, 0);
            if (in && rk < n_kv) {
                const uint16_t *src = static_cast<const uint16_t *>(is_k ? a.k : a.v) +
                                      (is_k ? t * a.k_s0 + hk * a.k_s1 : t * a.v_s0 + hk * a.v_s1) + da;
                wa[kQRows] = *reinterpret_cast<const uint2 *>(src);
                wb[kQRows] = *reinterpret_cast<const uint2 *>(src + (db - da));
            }
            if (rq == row0 && live && turns) {  // the token's angles, behind its first rows
                const float *cs = a.cs + static_cast<int64_t>(len - 1) * a.cs_s0 + 4 * lane;
                c = *reinterpret_cast<const float4 *>(cs);
                s = *reinterpret_cast<const float4 *>(cs + half);
            }
            if (wq < a.Hq) {
                factors(weights[0], c, s, own, cross);
#pragma unroll
                for (int i = 0; i < kQRows; ++i) {
                    const int r = rq + i * groups;
                    const uint64_t x[4] = {widen2<kBf16>(wa[i].x), widen2<kBf16>(wa[i].y), widen2<kBf16>(wb[i].x),
                                           widen2<kBf16>(wb[i].y)};
                    uint64_t y[4];
                    turn(x, norm_q, y);
                    if (!live) y[0] = y[1] = y[2] = y[3] = 0;
                    if (in && r < a.Hq) {
                        uint16_t *dst = oa + r * qo_s1;
                        store4<kBf16, false>(dst, y[0], y[1]);
                        store4<kBf16, false>(dst + (db - da), y[2], y[3]);
                    }
                }
            }
            const uint64_t x[4] = {widen2<kBf16>(wa[kQRows].x), widen2<kBf16>(wa[kQRows].y), widen2<kBf16>(wb[kQRows].x),
                                   widen2<kBf16>(wb[kQRows].y)};
            uint64_t y[4];
            factors(weights[1], c, s, own, cross);
            turn(x, norm_k, y);
            if (stored && rk < n_kv) {
                const float scale = is_k ? a.k_inv : a.v_inv;
                const uint64_t scale2 = pair(scale, scale);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = mul2(is_k ? y[e] : x[e], scale2);
                uint8_t *dst = static_cast<uint8_t *>(is_k ? a.kc : a.vc) +
                               ((is_k ? slot * a.kc_s0 + hk * a.kc_s1 : slot * a.vc_s0 + hk * a.vc_s1) + da) * ces;
                store4<kBf16, kF8>(dst, y[0], y[1]);
                store4<kBf16, kF8>(dst + (db - da) * ces, y[2], y[3]);
            }
        }
    }
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

// Covers 16-bit inputs of head dim 64, 128 or 256 with aligned contiguous
// rows, an output of their type, caches of their type or E4M3, and rotary dims
// in whole lanes; anything else: *used stays false.
cudaError_t launch_store_vec(const StoreArgs &a, cudaStream_t stream, bool *used) {
    *used = false;
    if (a.in_dt == SPD_F32 || a.qo_dt != a.in_dt || (a.c_dt != a.in_dt && a.c_dt != SPD_E4M3)) return cudaSuccess;
    if ((a.Hq - 1) * (a.q_s1 > 0 ? a.q_s1 : -a.q_s1) > INT32_MAX || (a.Hq - 1) * a.qo_s1 > INT32_MAX) return cudaSuccess;
    if (a.D != 64 && a.D != 128 && a.D != 256) return cudaSuccess;
    if (a.Rd % 8 != 0) return cudaSuccess;
    // base and row strides whole multiples of what a lane moves at a time
    auto rows_ok = [](const void *p, int bytes, int es, int64_t s0, int64_t s1, int64_t s2) {
        return s2 == 1 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s0 * es) % bytes == 0 && (s1 * es) % bytes == 0;
    };
    const int ces = a.c_dt == SPD_E4M3 ? 1 : 2;
    if (!rows_ok(a.q, 8, 2, a.q_s0, a.q_s1, a.q_s2) || !rows_ok(a.k, 8, 2, a.k_s0, a.k_s1, a.k_s2) ||
        !rows_ok(a.qo, 8, 2, a.qo_s0, a.qo_s1, a.qo_s2) || !rows_ok(a.kc, 4 * ces, ces, a.kc_s0, a.kc_s1, a.kc_s2) ||
        !rows_ok(a.cs, 16, 4, a.cs_s0, 0, a.cs_s1))
        return cudaSuccess;
    if (a.v != nullptr &&
        (!rows_ok(a.v, 8, 2, a.v_s0, a.v_s1, a.v_s2) || !rows_ok(a.vc, 4 * ces, ces, a.vc_s0, a.vc_s1, a.vc_s2)))
        return cudaSuccess;
    const int lanes = a.D / 8, n_kv = a.Hkv * (a.v != nullptr ? 2 : 1);
    // as many row groups to a token as its rows can use
    const int most = n_kv > (a.Hq + kQRows - 1) / kQRows ? n_kv : (a.Hq + kQRows - 1) / kQRows;
    int groups = 1;
    while (groups < most && groups < kVecThreads / lanes) groups *= 2;
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
