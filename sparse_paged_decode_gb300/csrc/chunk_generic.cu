// chunk_generic.cu -- the prefill attention calls on CUDA cores, for every
// type, head dim and stride that the calls accept.
//
// One CTA per (query token, kv head): the token's G query heads share every
// key.  A block of 128 keys at a time, one thread per key for the logits,
// then one thread per output dim for the products with V; the running
// maximum, the row sum and the accumulators stay in fp32.  Only keys that the
// token reads are loaded, so nothing that another slot holds can reach it.
#include <math.h>

#include "serve.cuh"
#include "spd_dispatch.h"
#include "spd_internal.cuh"

namespace spd {

namespace {

constexpr int kThreads = kBlock;  // one thread per key of a block
constexpr int kDimsPerThread = kMaxD / kThreads;

__global__ void __launch_bounds__(kThreads) chunk_generic_kernel(const ChunkArgs a) {
    __shared__ float qs[kMaxGroup][kMaxD];
    __shared__ float ps[kMaxGroup][kBlock];
    __shared__ float m_run[kMaxGroup], alpha_s[kMaxGroup], l_run[kMaxGroup];
    __shared__ uint32_t chosen[kMaxNB / 32];

    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x;
    const int G = a.Hq / a.Hkv;
    const int b = owning_sequence(a.cu, a.cu_s0, a.B, t);
    int32_t L = 0;
    const int32_t *row_ids = nullptr;  // the token's row of topk_idx
    int64_t bt_row = 0;
    if (b >= 0) {
        const int64_t i = t - a.cu[b * a.cu_s0];
        L = chunk_limit(a, b, i);
        if (L > 0) bt_row = a.sid[b * a.sid_s0] * a.bt_s0;
        if (a.tk != nullptr) {
            const int64_t row = static_cast<int64_t>(a.cub[b * a.cub_s0]) + i / a.bsq;
            if (row >= 0 && row < a.n_rows && row < a.cub[(b + 1) * a.cub_s0])
                row_ids = a.tk + h * a.tk_s0 + row * a.tk_s1;
            else
                L = 0;
        }
    }
    for (int i = tid; i < G * a.D; i += kThreads) {
        const int g = i / a.D, d = i % a.D;
        qs[g][d] = load_float(a.q, a.q_dt, t * a.q_s0 + (h * G + g) * a.q_s1 + d * a.q_s2);
    }
    if (tid < kMaxNB / 32) chosen[tid] = a.tk == nullptr ? 0xffffffffu : 0u;
    if (tid < kMaxGroup) {
        m_run[tid] = -INFINITY;
        l_run[tid] = 0.f;
    }
    __syncthreads();
    if (row_ids != nullptr && L > 0) {
        for (int k = tid; k < a.K; k += kThreads) {
            const int32_t id = row_ids[k * a.tk_s2];
            if (id >= 0 && id < a.NB) atomicOr(&chosen[id >> 5], 1u << (id & 31));
        }
    }
    __syncthreads();

    const float zscale = a.sm_scale * a.k_scale;
    float acc[kDimsPerThread][kMaxGroup];
#pragma unroll
    for (int c = 0; c < kDimsPerThread; ++c)
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) acc[c][g] = 0.f;
    bool any = false;  // the token reads a key

    for (int kb = 0; kb * kBlock < L; ++kb) {
        if (!((chosen[kb >> 5] >> (kb & 31)) & 1u)) continue;
        const int64_t page = a.bt[bt_row + kb * a.bt_s1];
        if (page < 0 || page >= a.P) continue;
        any = true;
        const int64_t base = page * kBlock;
        const float zs = zscale * page_k_scale(a.sc, page, h), vs = page_v_scale(a.sc, page, h);
        const int n_valid = min(kBlock, L - kb * kBlock);
        if (tid < n_valid) {
            const int64_t krow = (base + tid) * a.k_s0 + h * a.k_s1;
            float z[kMaxGroup];
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g) z[g] = 0.f;
            for (int d = 0; d < a.D; ++d) {
                const float kd = kv_value(a.k, a.kv_dt, krow + d);
#pragma unroll
                for (int g = 0; g < kMaxGroup; ++g)
                    if (g < G) z[g] = fmaf(qs[g][d], kd, z[g]);
            }
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g)
                if (g < G) ps[g][tid] = z[g] * zs;
        }
        __syncthreads();
        if (tid < G) {
            float bm = -INFINITY;
            for (int i = 0; i < n_valid; ++i) bm = fmaxf(bm, ps[tid][i]);
            const float m_new = fmaxf(m_run[tid], bm);
            alpha_s[tid] = (m_run[tid] == -INFINITY) ? 0.f : expf(m_run[tid] - m_new);
            m_run[tid] = m_new;
        }
        __syncthreads();
        if (tid < n_valid)
            // logits of -inf weigh nothing, also where the row has no others yet
            for (int g = 0; g < G; ++g) ps[g][tid] = ps[g][tid] == -INFINITY ? 0.f : expf(ps[g][tid] - m_run[g]);
        __syncthreads();
        if (tid < G) {
            float s = 0.f;
            for (int i = 0; i < n_valid; ++i) s += ps[tid][i];
            l_run[tid] = (alpha_s[tid] == 0.f ? 0.f : l_run[tid] * alpha_s[tid]) + s;
        }
#pragma unroll
        for (int c = 0; c < kDimsPerThread; ++c) {
            const int d = tid + c * kThreads;
            if (d >= a.D) continue;
            float part[kMaxGroup];
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g) part[g] = 0.f;
            for (int i = 0; i < n_valid; ++i) {
                const float vd = kv_value(a.v, a.kv_dt, (base + i) * a.v_s0 + h * a.v_s1 + d);
#pragma unroll
                for (int g = 0; g < kMaxGroup; ++g)
                    if (g < G) part[g] = fmaf(ps[g][i], vd, part[g]);
            }
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g)
                if (g < G) acc[c][g] = fmaf(acc[c][g], alpha_s[g], part[g] * vs);
        }
        __syncthreads();
    }

#pragma unroll
    for (int c = 0; c < kDimsPerThread; ++c) {
        const int d = tid + c * kThreads;
        if (d >= a.D) continue;
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= G) continue;
            const float o = any ? acc[c][g] * a.v_scale / l_run[g] : 0.f;
            static_cast<__nv_bfloat16 *>(a.out)[t * a.o_s0 + (h * G + g) * a.o_s1 + d * a.o_s2] =
                __float2bfloat16_rn(o);
        }
    }
}

}  // namespace

cudaError_t launch_chunk_generic(const ChunkArgs &a, cudaStream_t stream) {
    count_launches(1);
    chunk_generic_kernel<<<dim3(static_cast<unsigned>(a.total_q), static_cast<unsigned>(a.Hkv)), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace spd
