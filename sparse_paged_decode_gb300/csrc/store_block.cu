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

// The layouts of the vector store (store.cuh), one launch: the first CTAs append K
// and V, the others write the queries as store_vec_kernel does (in turn with the
// appending ones they took the same time).
//
// An appending CTA takes one K or V head of `tile` batch rows: the runs that
// begin in them, with the rows behind the tile that end the last one.  Runs are
// found by ballots over "row i does not continue row i - 1".  Then it goes from
// run to run, as many at a time as have kKept rows together: its warps take the
// rows in turn, whatever run they belong to, leave them in shared memory (K in
// fp32, V as it came) and bring each run's largest magnitude together by an atomic
// maximum (of the bits of numbers that are not negative: no order matters); one
// thread a run fixes its scale; the rows are rounded and stored from shared
// memory.  Held codes that grow are multiplied by the whole CTA behind that (16 KB
// a run at most: one round trip).
//
// Measured, 64 + 8 + 8 rows of 128 dims a token, called one by one (graph of calls
// in brackets): 8192 tokens 80.4 (78.1) us, 0.6 of the measured copy rate; 476
// rows of 64 requests 11.2 (9.1) us; 16 requests of a token 6.2 (3.7) us.  The
// queries alone take 54 us of the 8192 tokens, the appending alone 32: warps that
// wait bound it (24 an SM; issue on 49 % of the cycles, DRAM at 45 %).  One warp a
// short run and rows read twice took 84 us, rows kept in registers and 128
// registers a thread 96, four rows in flight instead of two 83.
constexpr int kMaxTile = 128;
constexpr int kKept = kBlock;  // rows kept in shared memory: a whole page's run

struct Append {
    int32_t slot[kVecThreads];              // of row tile0 - 1 + i; -1 where it stores nothing
    int32_t len[kVecThreads];
    uint32_t begins[kVecThreads / 32];      // bit per row: it does not continue the row before
    uint32_t leads[kVecThreads / 32];       // it begins a run of this tile
    uint32_t top[kMaxTile + 1];             // by the row that begins the run: its largest magnitude's bits,
    float inv[kMaxTile + 1];                // its scale's reciprocal
    int n_grown;
    int32_t grown[kMaxTile];                // runs whose pages hold codes that grow,
    float ratio[kMaxTile];                  // and by what
};

// The larger of two pairs' magnitudes, each half for itself.
template <bool kBf16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    if (kBf16) {
        const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162 *>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2 *>(&a)), __habs2(*reinterpret_cast<const __half2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// The largest finite magnitude of eight values.  A maximum passes NaN over; only
// where an infinity comes out are the values looked at one by one.
__device__ __forceinline__ float largest(const uint64_t (&y)[4]) {
    float v[8], top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) unpair(y[e], v[2 * e], v[2 * e + 1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
    if (top == INFINITY) {
        top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_abs(v[e]));
    }
    return top;
}

template <bool kBf16, int kLanes, int kMode, bool kIsK>
__device__ __forceinline__ void append_tile(const StoreArgs &a, const float *weights, Append &sh, uint4 *kept, int64_t tile0,
                                            int tile, int h) {
    constexpr int kWarps = kVecThreads / 32, kRows = 32 / kLanes;  // rows of a warp at a time
    constexpr int kStep = kWarps * kRows;                          // of the CTA
    constexpr int kBatch = kIsK ? 2 : 4;                           // such steps in flight (K has angles too)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = threadIdx.x % kLanes;
    const uint16_t *src = static_cast<const uint16_t *>(kIsK ? a.k : a.v) + h * (kIsK ? a.k_s1 : a.v_s1);
    const int64_t src_s0 = kIsK ? a.k_s0 : a.v_s0;
    uint8_t *dst = static_cast<uint8_t *>(kIsK ? a.kc : a.vc) + h * (kIsK ? a.kc_s1 : a.vc_s1);  // slot 0
    const int64_t dst_s0 = kIsK ? a.kc_s0 : a.vc_s0;
    float *scale_at = nullptr;  // of the run that this thread's row begins
    float old = 0.f;
    {
        const int i = threadIdx.x;
        const int64_t t = tile0 - 1 + i;
        Row r{0, -1, false, false};
        if (t >= 0 && t < a.T) r = row_of(a, t);
        const int32_t slot = r.stored ? r.slot : -1;
        sh.slot[i] = slot;
        sh.len[i] = r.len;
        if (i <= kMaxTile) sh.top[i] = 0;
        if (i == 0) sh.n_grown = 0;
        __syncthreads();
        const bool begins = !(i > 0 && slot >= 0 && slot % kBlock != 0 && sh.slot[i - 1] == slot - 1);
        const bool leads = begins && slot >= 0 && i >= 1 && i <= tile;
        if (leads) {
            scale_at = (kIsK ? a.ks + h * a.ks_s1 : a.vs + h * a.vs_s1) + slot / kBlock * (kIsK ? a.ks_s0 : a.vs_s0);
            if (slot % kBlock != 0) old = *scale_at;
        }
        const uint32_t b = __ballot_sync(0xffffffffu, begins), l = __ballot_sync(0xffffffffu, leads);
        if (lane == 0) {
            sh.begins[warp] = b;
            sh.leads[warp] = l;
        }
        __syncthreads();
    }
    // the rows from the first run's beginning to the last one's end
    int first = kVecThreads, end = 0;
#pragma unroll
    for (int w = 0; w <= kMaxTile / 32; ++w) {
        const uint32_t l = sh.leads[w];
        if (l == 0) continue;
        first = min(first, w * 32 + __ffs(l) - 1);
        end = w * 32 + 31 - __clz(l);
    }
    if (end == 0) {
        __syncthreads();  // before another tile's rows
        return;
    }
    {
        int w = end >> 5;
        uint32_t behind = sh.begins[w] & ~((2u << (end & 31)) - 1u);
        while (behind == 0 && ++w < kWarps) behind = sh.begins[w];
        end = behind != 0 ? w * 32 + __ffs(behind) - 1 : kVecThreads;
    }
    // the last row up to i that begins something (row 0 does)
    auto begin_of = [&](int i) {
        int w = i >> 5;
        uint32_t before = sh.begins[w] & ((2u << (i & 31)) - 1u);
        while (before == 0) before = sh.begins[--w];
        return w * 32 + 31 - __clz(before);
    };

    const RowLane<kLanes, kMode> me(a, col);
    const int da = kIsK ? me.da : 8 * col, db = kIsK ? me.db : da + 4;
    const int sub = warp * kRows + lane / kLanes;
    const bool wide = ((reinterpret_cast<uintptr_t>(dst) | static_cast<uintptr_t>(dst_s0)) & 7) == 0;
    for (int lo = first, hi; lo < end; lo = hi) {
        // whole runs: a run has at most kKept rows, so one fits
        hi = end - lo <= kKept ? end : begin_of(lo + kKept);
        const bool one = begin_of(hi - 1) == lo;  // a long run's rows by themselves, the common case of a chunk
        float acc = 0.f;
        for (int i0 = lo; i0 < hi; i0 += kStep * kBatch) {
            // all loads of the turn, then the mathematics; a row that is not there is
            // made of zeros
            uint2 wa[kBatch], wb[kBatch];
            float4 c[kBatch], s[kBatch];
            bool there[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + sub + k * kStep;
                there[k] = i < hi && (one || sh.slot[i] >= 0);
                wa[k] = wb[k] = make_uint2(0, 0);
                c[k] = make_float4(1.f, 1.f, 1.f, 1.f);
                s[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (there[k]) {
                    const uint16_t *row = src + (tile0 - 1 + i) * src_s0 + da;
                    wa[k] = *reinterpret_cast<const uint2 *>(row);
                    wb[k] = *reinterpret_cast<const uint2 *>(row + (db - da));
                    if (kIsK && me.turns) {
                        const float *cs = a.cs + static_cast<int64_t>(sh.len[i] - 1) * a.cs_s0 + 4 * col;
                        c[k] = *reinterpret_cast<const float4 *>(cs);
                        s[k] = *reinterpret_cast<const float4 *>(cs + a.Rd / 2);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + sub + k * kStep;
                float top;
                if (kIsK) {
                    const uint64_t x[4] = {widen2<kBf16>(wa[k].x), widen2<kBf16>(wa[k].y), widen2<kBf16>(wb[k].x),
                                           widen2<kBf16>(wb[k].y)};
                    uint64_t own[4], cross[4], y[4];
                    me.factors(weights, c[k], s[k], own, cross);
                    me.turn(x, own, cross, a.wk != nullptr, a.eps, y);
                    top = largest(y);
                    if (there[k]) {
                        ulonglong2 *row = reinterpret_cast<ulonglong2 *>(kept) + (i - lo) * (2 * kLanes);
                        row[da / 4] = make_ulonglong2(y[0], y[1]);
                        row[db / 4] = make_ulonglong2(y[2], y[3]);
                    }
                } else {
                    const uint32_t m = max_abs2<kBf16>(max_abs2<kBf16>(wa[k].x, wa[k].y), max_abs2<kBf16>(wb[k].x, wb[k].y));
                    float t0, t1;
                    unpair(widen2<kBf16>(m), t0, t1);
                    top = fmaxf(t0, t1);
                    if (!(top < INFINITY)) {
                        const uint64_t x[4] = {widen2<kBf16>(wa[k].x), widen2<kBf16>(wa[k].y), widen2<kBf16>(wb[k].x),
                                               widen2<kBf16>(wb[k].y)};
                        top = largest(x);
                    }
                    if (there[k]) kept[(i - lo) * kLanes + col] = make_uint4(wa[k].x, wa[k].y, wb[k].x, wb[k].y);
                }
                if (one) {
                    acc = fmaxf(acc, top);
                } else {
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                    if (there[k] && col == 0) atomicMax(&sh.top[begin_of(i)], __float_as_uint(top));
                }
            }
        }
        if (one) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) acc = fmaxf(acc, __shfl_xor_sync(0xffffffffu, acc, m));
            if (lane == 0) atomicMax(&sh.top[lo], __float_as_uint(acc));
        }
        __syncthreads();
        if (scale_at != nullptr && threadIdx.x >= lo && threadIdx.x < hi) {
            float ratio;
            const float scale = page_scale(__uint_as_float(sh.top[threadIdx.x]), old, ratio);
            *scale_at = scale;
            sh.inv[threadIdx.x] = 1.f / scale;
            if (ratio != 1.f) {
                const int k = atomicAdd(&sh.n_grown, 1);
                sh.grown[k] = threadIdx.x;
                sh.ratio[k] = ratio;
            }
        }
        __syncthreads();
        // a lane rounds and stores eight neighbouring dims
        for (int i = lo + sub; i < hi; i += kStep) {
            const int32_t slot = sh.slot[i];
            if (slot < 0) continue;
            const float inv = sh.inv[one ? lo : begin_of(i)];
            const uint64_t inv2 = pair(inv, inv);
            uint64_t y[4];
            if (kIsK) {
                const ulonglong2 *row = reinterpret_cast<const ulonglong2 *>(kept) + (i - lo) * (2 * kLanes) + 2 * col;
                y[0] = row[0].x, y[1] = row[0].y, y[2] = row[1].x, y[3] = row[1].y;
            } else {
                const uint4 w = kept[(i - lo) * kLanes + col];
                y[0] = widen2<kBf16>(w.x), y[1] = widen2<kBf16>(w.y), y[2] = widen2<kBf16>(w.z), y[3] = widen2<kBf16>(w.w);
            }
            const uint32_t c0 = e4m3x4(mul2(y[0], inv2), mul2(y[1], inv2)), c1 = e4m3x4(mul2(y[2], inv2), mul2(y[3], inv2));
            uint8_t *at = dst + slot * dst_s0 + 8 * col;
            if (wide) {
                *reinterpret_cast<uint2 *>(at) = make_uint2(c0, c1);
            } else {
                reinterpret_cast<uint32_t *>(at)[0] = c0;
                reinterpret_cast<uint32_t *>(at)[1] = c1;
            }
        }
        __syncthreads();  // before other rows take their place
    }
    for (int g = 0; g < sh.n_grown; ++g) {
        constexpr int kWords = 2 * kLanes, kFlight = 8;  // words of a row; of a thread in flight
        const int32_t slot = sh.slot[sh.grown[g]];
        const int words = slot % kBlock * kWords;
        const float ratio = sh.ratio[g];
        uint8_t *page = dst + static_cast<int64_t>(slot / kBlock * kBlock) * dst_s0;
        auto at = [&](int i) { return reinterpret_cast<uint32_t *>(page + i / kWords * dst_s0) + i % kWords; };
        for (int i0 = threadIdx.x; i0 < words; i0 += kFlight * kVecThreads) {
            uint32_t w[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) w[k] = i0 + k * kVecThreads < words ? *at(i0 + k * kVecThreads) : 0u;
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                uint32_t out = 0;
#pragma unroll
                for (int b = 0; b < 32; b += 8) out |= static_cast<uint32_t>(rescaled((w[k] >> b) & 0xffu, ratio)) << b;
                if (i0 + k * kVecThreads < words) *at(i0 + k * kVecThreads) = out;
            }
        }
    }
    __syncthreads();  // before another tile's rows
}

template <bool kBf16, int kLanes, int kMode>
__global__ void __launch_bounds__(kVecThreads, kVecCtas)
store_block_vec_kernel(const StoreArgs a, int groups, int tile, int64_t items, unsigned kv_blocks) {
    __shared__ __align__(16) float weights[2][8 * kLanes];
    __shared__ Append sh;
    extern __shared__ uint4 kept[];  // kKept rows of 8 * kLanes floats
    load_weights<kLanes>(a, weights);
    if (blockIdx.x >= kv_blocks) {
        store_rows<kBf16, true, kLanes, kMode, false>(a, weights, groups, blockIdx.x - kv_blocks, gridDim.x - kv_blocks);
        return;
    }
    const int n_heads = 2 * a.Hkv;
    for (int64_t item = blockIdx.x; item < items; item += kv_blocks) {
        const int u = static_cast<int>(item % n_heads);
        const int64_t tile0 = item / n_heads * tile;
        if (u < a.Hkv) append_tile<kBf16, kLanes, kMode, true>(a, weights[1], sh, kept, tile0, tile, u);
        else append_tile<kBf16, kLanes, kMode, false>(a, weights[1], sh, kept, tile0, tile, u - a.Hkv);
    }
}

template <bool kBf16, int kLanes>
cudaError_t launch_block_vec(const StoreArgs &a, unsigned grid, int groups, int tile, int64_t items, unsigned kv_blocks,
                             cudaStream_t stream) {
    auto kernel = a.interleaved    ? store_block_vec_kernel<kBf16, kLanes, 2>
                  : a.Rd == a.D    ? store_block_vec_kernel<kBf16, kLanes, 0>
                                   : store_block_vec_kernel<kBf16, kLanes, 1>;
    constexpr int kSmem = kKept * 8 * kLanes * sizeof(float);
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kVecThreads, kSmem, stream>>>(a, groups, tile, items, kv_blocks);
    return cudaGetLastError();
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
    // rows of a tile: so many that the appending CTAs are two to an SM, in powers of
    // two (476 rows: 9.1 us with two, 10.4 with four, 12.6 with eight; 1999 rows of
    // chunks 23.5, 24.2, 25.8)
    const int64_t per_cta = static_cast<int64_t>(a.T) * 2 * a.Hkv / (2 * device_sm_count());
    int tile = 8;
    while (tile < kMaxTile && tile < per_cta) tile *= 2;
    const int64_t items = (static_cast<int64_t>(a.T) + tile - 1) / tile * 2 * a.Hkv;
    const unsigned kv_blocks = static_cast<unsigned>(items < 16 * room ? items : 16 * room);
    const int tokens = kVecThreads / lanes / groups;
    const int64_t want = (static_cast<int64_t>(a.T) + tokens - 1) / tokens;
    // as many query CTAs as there are places beside the appending ones, or a few
    // rounds of them: what one takes is to be short next to the call (8192 tokens:
    // 84.8 us with one round, 80.3 with two, 78 with four, 79 with eight)
    const int64_t beside = room > 2 * static_cast<int64_t>(kv_blocks) ? room - kv_blocks : 4 * room;
    const unsigned grid = kv_blocks + static_cast<unsigned>(want < beside ? want : beside);
    const bool bf16 = a.in_dt == SPD_BF16;
    const auto launch = lanes == 8    ? (bf16 ? launch_block_vec<true, 8> : launch_block_vec<false, 8>)
                        : lanes == 16 ? (bf16 ? launch_block_vec<true, 16> : launch_block_vec<false, 16>)
                                      : (bf16 ? launch_block_vec<true, 32> : launch_block_vec<false, 32>);
    const cudaError_t e = launch(a, grid, groups, tile, items, kv_blocks, stream);
    if (e != cudaSuccess) return e;
    count_launches(1);
    *used = true;
    return cudaSuccess;
}

}  // namespace spd
