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

// The scale of a page and head whose new rows reach `top` and whose scale was
// `old` (0 where the page is begun anew), and what its held codes are multiplied
// by: 1 where they stay as they are.
__device__ __forceinline__ float page_scale(float top, float old, float &ratio) {
    const float need = scale_of(top);
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
        const float scale = page_scale(top, f > 0 ? *at : 0.f, ratio), inv = 1.f / scale;
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

// The layouts of the vector store (store.cuh), one launch: the first kv_blocks
// CTAs append K and V, the others write the queries as store_vec_kernel does.
//
// An appending CTA takes one K or V head of `tile` batch rows: the runs that
// begin in them, with the rows behind the tile that end the last one.  Runs are
// found by ballots over "row i does not continue row i - 1".  A run of more than
// kShort rows is the whole CTA's work, a shorter one a warp's, and held codes
// that grow are multiplied by the whole CTA behind all runs (16 KB at most: one
// round trip).  Rows are read twice, for their maximum and to be stored: the
// second time they come from L1 or L2, and nothing is kept between.
constexpr int kShort = 16;
constexpr int kMaxTile = 128;

struct Append {
    int32_t slot[kVecThreads];              // of row tile0 - 1 + i; -1 where it stores nothing
    uint32_t begins[kVecThreads / 32];      // bit per row: it does not continue the row before
    uint32_t leads[kVecThreads / 32];       // it begins a run of this tile
    float top[kVecThreads / 32];
    int n_grown;
    int32_t grown[kMaxTile];                // rows of short runs whose pages grow,
    float ratio[kMaxTile];                  // and by what
};

// What the appending of one head works on.
template <bool kBf16, int kLanes, int kMode>
struct Head {
    const StoreArgs &a;
    const float *weights;                   // of K
    const RowLane<kLanes, kMode> me;
    const bool is_k, norm;
    const int h, lane;                      // kv head, lane within a row's lanes
    const uint16_t *src;
    int64_t src_s0;
    uint8_t *dst;                           // head h of slot 0
    int64_t dst_s0;

    __device__ __forceinline__ Head(const StoreArgs &a_, const float *w, bool k, int h_)
        : a(a_), weights(w), me(a_, threadIdx.x % kLanes), is_k(k), norm(k && a_.wk != nullptr), h(h_),
          lane(threadIdx.x % kLanes) {
        src = static_cast<const uint16_t *>(is_k ? a.k : a.v) + h * (is_k ? a.k_s1 : a.v_s1);
        src_s0 = is_k ? a.k_s0 : a.v_s0;
        dst = static_cast<uint8_t *>(is_k ? a.kc : a.vc) + h * (is_k ? a.kc_s1 : a.vc_s1);
        dst_s0 = is_k ? a.kc_s0 : a.vc_s0;
    }

    // Rows t + j0, t + j0 + step, ... of a run of n rows, kBatch of them at a time
    // (all loads, then the mathematics): f(j, y) for the row's values y.  Lanes
    // whose row lies behind the run work on zeros, and get no call.
    template <typename F>
    __device__ __forceinline__ void rows(int64_t t, int n, int warp_row, int step, F &&f) const {
        constexpr int kBatch = 2;
        const int sub = threadIdx.x % 32 / kLanes;
        for (int j0 = warp_row; j0 < n; j0 += kBatch * step) {  // the same for a warp's lanes
            uint2 wa[kBatch], wb[kBatch];
            float4 c[kBatch], s[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * step + sub;
                wa[i] = wb[i] = make_uint2(0, 0);
                c[i] = make_float4(1.f, 1.f, 1.f, 1.f);
                s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < n) {
                    const uint16_t *row = src + (t + j) * src_s0 + me.da;
                    wa[i] = *reinterpret_cast<const uint2 *>(row);
                    wb[i] = *reinterpret_cast<const uint2 *>(row + (me.db - me.da));
                    if (is_k && me.turns) {
                        const float *cs = a.cs + static_cast<int64_t>(a.tl[(t + j) * a.tl_s0] - 1) * a.cs_s0 + 4 * lane;
                        c[i] = *reinterpret_cast<const float4 *>(cs);
                        s[i] = *reinterpret_cast<const float4 *>(cs + a.Rd / 2);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * step + sub;
                const uint64_t x[4] = {widen2<kBf16>(wa[i].x), widen2<kBf16>(wa[i].y), widen2<kBf16>(wb[i].x),
                                       widen2<kBf16>(wb[i].y)};
                uint64_t y[4] = {x[0], x[1], x[2], x[3]};
                if (is_k) {  // the same for the whole CTA
                    uint64_t own[4], cross[4];
                    me.factors(weights, c[i], s[i], own, cross);
                    me.turn(x, own, cross, norm, a.eps, y);
                }
                if (j < n) f(j, y);
            }
        }
    }

    __device__ __forceinline__ float largest(int64_t t, int n, int warp_row, int step) const {
        float top = 0.f;
        rows(t, n, warp_row, step, [&](int, const uint64_t *y) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo, hi;
                unpair(y[e], lo, hi);
                top = fmaxf(top, fmaxf(finite_abs(lo), finite_abs(hi)));
            }
        });
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        return top;
    }

    __device__ __forceinline__ void keep(int64_t t, int n, int32_t slot, float scale, int warp_row, int step) const {
        const float inv = 1.f / scale;
        const uint64_t inv2 = pair(inv, inv);
        rows(t, n, warp_row, step, [&](int j, const uint64_t *y) {
            uint8_t *at = dst + (static_cast<int64_t>(slot) + j) * dst_s0 + me.da;
            store4<kBf16, true>(at, mul2(y[0], inv2), mul2(y[1], inv2));
            store4<kBf16, true>(at + (me.db - me.da), mul2(y[2], inv2), mul2(y[3], inv2));
        });
    }

    // the f codes rows that a page holds, times ratio; the whole CTA
    __device__ __forceinline__ void grow(int64_t page, int f, float ratio) const {
        constexpr int kWords = 2 * kLanes, kBatch = 8;  // words of a row; of a thread at a time
        for (int i0 = threadIdx.x; i0 < f * kWords; i0 += kBatch * kVecThreads) {
            uint32_t w[kBatch];
            auto at = [&](int i) {
                return reinterpret_cast<uint32_t *>(dst + (page * kBlock + i / kWords) * dst_s0) + i % kWords;
            };
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k * kVecThreads < f * kWords) w[k] = *at(i0 + k * kVecThreads);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k * kVecThreads < f * kWords) {
                    uint32_t out = 0;
#pragma unroll
                    for (int b = 0; b < 32; b += 8) out |= static_cast<uint32_t>(rescaled((w[k] >> b) & 0xffu, ratio)) << b;
                    *at(i0 + k * kVecThreads) = out;
                }
        }
    }
};

template <bool kBf16, int kLanes, int kMode>
__device__ __forceinline__ void append_tile(const StoreArgs &a, const float *weights, Append &sh, int64_t tile0, int tile,
                                            bool is_k, int h) {
    constexpr int kWarps = kVecThreads / 32, kRows = 32 / kLanes;  // rows of a warp at a time
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = threadIdx.x;
    {
        const int64_t t = tile0 - 1 + i;
        int32_t slot = -1;
        if (t >= 0 && t < a.T) {
            const Row r = row_of(a, t);
            if (r.stored) slot = r.slot;
        }
        sh.slot[i] = slot;
        if (i == 0) sh.n_grown = 0;
        __syncthreads();
        const bool continues = i > 0 && slot >= 0 && slot % kBlock != 0 && sh.slot[i - 1] == slot - 1;
        const uint32_t begins = __ballot_sync(0xffffffffu, !continues);
        const uint32_t leads = __ballot_sync(0xffffffffu, !continues && slot >= 0 && i >= 1 && i <= tile);
        if (lane == 0) {
            sh.begins[warp] = begins;
            sh.leads[warp] = leads;
        }
        __syncthreads();
    }
    const Head<kBf16, kLanes, kMode> head(a, weights, is_k, h);
    float *scales = is_k ? a.ks + h * a.ks_s1 : a.vs + h * a.vs_s1;
    const int64_t scales_s0 = is_k ? a.ks_s0 : a.vs_s0;
    int n_short = 0;
    for (int w = 0; w * 32 <= tile; ++w) {
        for (uint32_t bits = sh.leads[w]; bits != 0; bits &= bits - 1) {
            const int at = w * 32 + __ffs(bits) - 1;
            // the run ends where the next row begins something
            int word = at >> 5;
            uint32_t behind = sh.begins[word] & ~((2u << (at & 31)) - 1u);
            while (behind == 0 && ++word < kWarps) behind = sh.begins[word];
            const int n = (behind != 0 ? word * 32 + __ffs(behind) - 1 : kVecThreads) - at;
            const bool whole = n > kShort;
            if (!whole && n_short++ % kWarps != warp) continue;
            const int32_t slot = sh.slot[at];
            const int64_t t = tile0 - 1 + at, page = slot / kBlock;
            const int f = slot % kBlock;
            float *scale_at = scales + page * scales_s0;
            const float old = f > 0 ? *scale_at : 0.f;
            const int row0 = whole ? warp * kRows : 0, step = whole ? kWarps * kRows : kRows;
            float top = head.largest(t, n, row0, step);
            if (whole) {
                if (lane == 0) sh.top[warp] = top;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sh.top[k]);
            }
            float ratio;
            const float scale = page_scale(top, old, ratio);
            if (lane == 0 && (!whole || warp == 0)) {
                *scale_at = scale;
                if (ratio != 1.f) {
                    const int k = atomicAdd(&sh.n_grown, 1);
                    sh.grown[k] = at;
                    sh.ratio[k] = ratio;
                }
            }
            head.keep(t, n, slot, scale, row0, step);
            if (whole) __syncthreads();  // before the next long run's maxima
        }
    }
    __syncthreads();
    for (int k = 0; k < sh.n_grown; ++k) {
        const int32_t slot = sh.slot[sh.grown[k]];
        head.grow(slot / kBlock, slot % kBlock, sh.ratio[k]);
    }
    __syncthreads();  // before another tile's rows
}

template <bool kBf16, int kLanes, int kMode>
__global__ void __launch_bounds__(kVecThreads, kVecCtas)
store_block_vec_kernel(const StoreArgs a, int groups, int tile, int64_t items, unsigned kv_blocks) {
    __shared__ __align__(16) float weights[2][8 * kLanes];
    __shared__ Append sh;
    load_weights<kLanes>(a, weights);
    if (blockIdx.x >= kv_blocks) {
        store_rows<kBf16, true, kLanes, kMode, false>(a, weights, groups, blockIdx.x - kv_blocks, gridDim.x - kv_blocks);
        return;
    }
    const int n_heads = 2 * a.Hkv;
    for (int64_t item = blockIdx.x; item < items; item += kv_blocks) {
        const int u = static_cast<int>(item % n_heads);
        append_tile<kBf16, kLanes, kMode>(a, weights[1], sh, item / n_heads * tile, tile, u < a.Hkv,
                                          u < a.Hkv ? u : u - a.Hkv);
    }
}

template <bool kBf16, int kLanes>
void launch_block_vec(const StoreArgs &a, unsigned grid, int groups, int tile, int64_t items, unsigned kv_blocks,
                      cudaStream_t stream) {
    auto kernel = a.interleaved    ? store_block_vec_kernel<kBf16, kLanes, 2>
                  : a.Rd == a.D    ? store_block_vec_kernel<kBf16, kLanes, 0>
                                   : store_block_vec_kernel<kBf16, kLanes, 1>;
    kernel<<<grid, kVecThreads, 0, stream>>>(a, groups, tile, items, kv_blocks);
}

}  // namespace

cudaError_t launch_store_block_generic(const StoreArgs &a, cudaStream_t stream) {
    count_launches(1);
    store_block_generic_kernel<<<static_cast<unsigned>(a.T), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

// Covers what the vector store covers; anything else: *used stays false.
cudaError_t launch_store_block_vec(const StoreArgs &a, cudaStream_t stream, bool *used) {
    *used = false;
    if (!store_vec_covers(a)) return cudaSuccess;
    const int lanes = a.D / 8, groups = store_row_groups(a, 1);
    const int64_t room = static_cast<int64_t>(device_sm_count()) * kVecCtas;
    // rows of a tile: so many that the appending CTAs are a few to an SM
    const int64_t per_cta = static_cast<int64_t>(a.T) * 2 * a.Hkv / (8 * device_sm_count());
    int tile = 8;
    while (tile < kMaxTile && tile < per_cta) tile *= 2;
    const int64_t items = (static_cast<int64_t>(a.T) + tile - 1) / tile * 2 * a.Hkv;
    const unsigned kv_blocks = static_cast<unsigned>(items < 16 * room ? items : 16 * room);
    const int tokens = kVecThreads / lanes / groups;
    const int64_t want = (static_cast<int64_t>(a.T) + tokens - 1) / tokens;
    const unsigned grid = kv_blocks + static_cast<unsigned>(want < room ? want : room);
    const bool bf16 = a.in_dt == SPD_BF16;
    if (lanes == 8) (bf16 ? launch_block_vec<true, 8> : launch_block_vec<false, 8>)(a, grid, groups, tile, items, kv_blocks, stream);
    else if (lanes == 16) (bf16 ? launch_block_vec<true, 16> : launch_block_vec<false, 16>)(a, grid, groups, tile, items, kv_blocks, stream);
    else (bf16 ? launch_block_vec<true, 32> : launch_block_vec<false, 32>)(a, grid, groups, tile, items, kv_blocks, stream);
    count_launches(1);
    *used = true;
    return cudaGetLastError();
}

}  // namespace spd
