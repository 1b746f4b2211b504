// spd_abi.cu -- the extern "C" entry points: host-side validation of every
// descriptor, the error channel, and dispatch to the kernels.
//
// Validation follows "Kernel ABI" -- Core rules (exact arguments, every
// output cell written honouring shape/dtype/stride, inputs unchanged, no
// output aliasing an input, stay inside the declared capability domain) and
// "Kernel ABI" -- Capability and fallback behavior (fail closed outside the
// domain).  Nothing here reads device memory or synchronises.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "prefill.cuh"
#include "sdpa.cuh"
#include "serve.cuh"
#include "spd_internal.cuh"
#include "spd_dispatch.h"

namespace spd {
namespace {

thread_local int g_status = SPD_OK;
thread_local char g_msg[512] = "ok";

void set_ok() {
    g_status = SPD_OK;
    snprintf(g_msg, sizeof g_msg, "ok");
}

bool fail(int code, const char *fmt, ...) {
    g_status = code;
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return false;
}

int elem_size(int dt) {
    switch (dt) {
    case SPD_F32: return 4;
    case SPD_BF16: return 2;
    case SPD_F16: return 2;
    case SPD_E4M3: return 1;
    case SPD_I32: return 4;
    default: return 0;
    }
}

const char *dtype_name(int dt) {
    switch (dt) {
    case SPD_F32: return "f32";
    case SPD_BF16: return "bf16";
    case SPD_F16: return "f16";
    case SPD_E4M3: return "e4m3";
    case SPD_I32: return "i32";
    default: return "?";
    }
}

int64_t numel(const spd_tensor *t) {
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

// Descriptor sanity: present, known dtype among `allowed`, rank, non-negative
// extents, aligned data pointer when the tensor is not empty.
bool check_desc(const spd_tensor *t, const char *name, int ndim, std::initializer_list<int> allowed) {
    if (t == nullptr) return fail(SPD_ERR_INVALID_ARGUMENT, "%s: descriptor is NULL", name);
    if (t->ndim != ndim)
        return fail(SPD_ERR_INVALID_ARGUMENT, "%s: expected %d dims, got %d", name, ndim, t->ndim);
    bool ok = false;
    for (int dt : allowed) ok = ok || (t->dtype == dt);
    if (!ok) return fail(SPD_ERR_UNSUPPORTED, "%s: dtype %s not supported here", name, dtype_name(t->dtype));
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] < 0) return fail(SPD_ERR_INVALID_ARGUMENT, "%s: negative extent in dim %d", name, i);
    if (numel(t) > 0) {
        if (t->data == nullptr) return fail(SPD_ERR_INVALID_ARGUMENT, "%s: data is NULL", name);
        if (reinterpret_cast<uintptr_t>(t->data) % elem_size(t->dtype) != 0)
            return fail(SPD_ERR_INVALID_ARGUMENT, "%s: data not aligned to its element size", name);
    }
    return true;
}

// Byte range [lo, hi) spanned by a non-empty tensor.
void byte_span(const spd_tensor *t, uintptr_t *lo, uintptr_t *hi) {
    int64_t mn = 0, mx = 0;
    for (int i = 0; i < t->ndim; ++i) {
        const int64_t ext = t->stride[i] * (t->shape[i] - 1);
        if (ext < 0) mn += ext; else mx += ext;
    }
    const int es = elem_size(t->dtype);
    *lo = reinterpret_cast<uintptr_t>(t->data) + mn * es;
    *hi = reinterpret_cast<uintptr_t>(t->data) + (mx + 1) * es;
}

// An output must map distinct cells to distinct elements: strictly positive
// strides on dims of extent > 1 that nest without overlap.
bool check_output_layout(const spd_tensor *t, const char *name) {
    int idx[4], n = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] <= 1) continue;
        if (t->stride[i] <= 0)
            return fail(SPD_ERR_INVALID_ARGUMENT, "%s: output strides must be positive", name);
        idx[n++] = i;
    }
    std::sort(idx, idx + n, [&](int x, int y) { return t->stride[x] < t->stride[y]; });
    int64_t span = 0;  // elements covered by the inner dims
    for (int j = 0; j < n; ++j) {
        const int i = idx[j];
        if (t->stride[i] <= span)
            return fail(SPD_ERR_ALIASING, "%s: output strides make cells overlap", name);
        span += t->stride[i] * (t->shape[i] - 1);
    }
    return true;
}

bool check_no_overlap(const spd_tensor *out, const char *oname, std::initializer_list<const spd_tensor *> ins) {
    if (numel(out) == 0) return true;
    uintptr_t olo, ohi;
    byte_span(out, &olo, &ohi);
    for (const spd_tensor *in : ins) {
        if (in == nullptr || numel(in) == 0) continue;
        uintptr_t ilo, ihi;
        byte_span(in, &ilo, &ihi);
        if (olo < ihi && ilo < ohi)
            return fail(SPD_ERR_ALIASING, "%s overlaps an input", oname);
    }
    return true;
}

bool check_scalar(float v, const char *name) {
    if (!(v == v) || v == INFINITY || v == -INFINITY)
        return fail(SPD_ERR_INVALID_ARGUMENT, "%s must be finite", name);
    return true;
}

// Shared metadata: block_table [R, NB], seq_lens [T], req_idx [T].
bool check_paging(const spd_tensor *bt, const spd_tensor *sl, const spd_tensor *ri, int64_t T,
                  int32_t block_size) {
    if (!check_desc(bt, "block_table", 2, {SPD_I32})) return false;
    if (!check_desc(sl, "seq_lens", 1, {SPD_I32})) return false;
    if (!check_desc(ri, "req_idx", 1, {SPD_I32})) return false;
    if (block_size != kBlock)
        return fail(SPD_ERR_UNSUPPORTED, "block_size must be %d (got %d)", kBlock, block_size);
    if (sl->shape[0] != T || ri->shape[0] != T)
        return fail(SPD_ERR_INVALID_ARGUMENT, "seq_lens and req_idx must have T=%lld entries", (long long)T);
    if (bt->shape[1] < 1 || bt->shape[1] > kMaxNB)
        return fail(SPD_ERR_UNSUPPORTED, "page-table capacity NB=%lld outside [1, %d]",
                    (long long)bt->shape[1], kMaxNB);
    if (T > 0 && bt->shape[0] < 1)
        return fail(SPD_ERR_INVALID_ARGUMENT, "block_table has no rows");
    return true;
}

// Scales [P, Hkv] of a block-scaled cache of P pages.
bool check_scales(const spd_tensor *t, const char *name, int64_t P, int64_t Hkv) {
    if (!check_desc(t, name, 2, {SPD_F32})) return false;
    if (t->shape[0] != P || t->shape[1] != Hkv)
        return fail(SPD_ERR_INVALID_ARGUMENT, "%s must be [pages=%lld, Hkv=%lld]", name, (long long)P, (long long)Hkv);
    return true;
}

PageScales page_scales(const spd_tensor *ks, const spd_tensor *vs) {
    PageScales s{};
    if (ks == nullptr) return s;
    // a cache without pages has no scales either: nothing reads them
    s.k = static_cast<const float *>(ks->data); s.k_s0 = ks->stride[0]; s.k_s1 = ks->stride[1];
    s.v = static_cast<const float *>(vs->data); s.v_s0 = vs->stride[0]; s.v_s1 = vs->stride[1];
    return s;
}

bool check_cuda(cudaError_t e, const char *what) {
    if (e != cudaSuccess)
        return fail(SPD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return true;
}

// ----------------------------------------------------------------- stage 1

bool block_score(const spd_tensor *q, const spd_tensor *k, const spd_tensor *bt, const spd_tensor *sl,
                 const spd_tensor *ri, int32_t block_size, const spd_tensor *out, float idx_scale,
                 cudaStream_t stream) {
    if (!check_desc(q, "q_idx", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(k, "k_idx_cache", 3, {SPD_F32, SPD_BF16, SPD_F16, SPD_E4M3})) return false;
    if (!check_desc(out, "scores", 3, {SPD_F32})) return false;
    const int64_t T = q->shape[0], Hi = q->shape[1], Di = q->shape[2];
    if (!check_paging(bt, sl, ri, T, block_size)) return false;
    if (k->dtype != q->dtype && k->dtype != SPD_E4M3)
        return fail(SPD_ERR_UNSUPPORTED, "k_idx_cache dtype must match q_idx (or be e4m3)");
    if (k->shape[1] != 1) return fail(SPD_ERR_UNSUPPORTED, "k_idx_cache must have one index key head");
    if (k->shape[2] != Di) return fail(SPD_ERR_INVALID_ARGUMENT, "k_idx_cache head dim != q_idx head dim");
    if (k->shape[0] % kBlock != 0) return fail(SPD_ERR_INVALID_ARGUMENT, "k_idx_cache slots not a whole number of pages");
    if (Di < 1 || Di > kMaxDi) return fail(SPD_ERR_UNSUPPORTED, "Di=%lld outside [1, %d]", (long long)Di, kMaxDi);
    if (Hi < 1 || Hi > 65535) return fail(SPD_ERR_UNSUPPORTED, "Hi=%lld outside [1, 65535]", (long long)Hi);
    const int64_t NB = bt->shape[1];
    if (out->shape[0] != Hi || out->shape[1] != T || out->shape[2] != NB)
        return fail(SPD_ERR_INVALID_ARGUMENT, "scores must be [Hi=%lld, T=%lld, NB=%lld]", (long long)Hi,
                    (long long)T, (long long)NB);
    if (T > INT32_MAX / 2) return fail(SPD_ERR_UNSUPPORTED, "T too large");
    if (!(idx_scale > 0.f) || idx_scale == INFINITY) return fail(SPD_ERR_UNSUPPORTED, "idx_scale must be finite and > 0");
    if (!check_output_layout(out, "scores")) return false;
    if (!check_no_overlap(out, "scores", {q, k, bt, sl, ri})) return false;
    if (T == 0) return true;

    ScoreArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = k->data; a.k_s0 = k->stride[0]; a.k_s2 = k->stride[2];
    a.bt = static_cast<const int32_t *>(bt->data); a.bt_s0 = bt->stride[0]; a.bt_s1 = bt->stride[1];
    a.sl = static_cast<const int32_t *>(sl->data); a.sl_s0 = sl->stride[0];
    a.ri = static_cast<const int32_t *>(ri->data); a.ri_s0 = ri->stride[0];
    a.out = static_cast<float *>(out->data); a.o_s0 = out->stride[0]; a.o_s1 = out->stride[1]; a.o_s2 = out->stride[2];
    a.q_dt = q->dtype; a.k_dt = k->dtype;
    a.T = (int32_t)T; a.Hi = (int32_t)Hi; a.Di = (int32_t)Di; a.R = (int32_t)bt->shape[0]; a.NB = (int32_t)NB;
    a.P = k->shape[0] / kBlock;
    a.idx_scale = idx_scale;
    return check_cuda(dispatch_score(a, stream), "msa_block_score launch");
}

// ----------------------------------------------------------------- stage 2

bool select_topk(const spd_tensor *s, const spd_tensor *o, cudaStream_t stream) {
    if (!check_desc(s, "scores", 3, {SPD_F32})) return false;
    if (!check_desc(o, "topk_idx", 3, {SPD_I32})) return false;
    const int64_t Hi = s->shape[0], T = s->shape[1], NB = s->shape[2], K = o->shape[2];
    if (o->shape[0] != Hi || o->shape[1] != T)
        return fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx must be [Hi, T, K] matching scores");
    if (NB < 1 || NB > kMaxNB) return fail(SPD_ERR_UNSUPPORTED, "NB=%lld outside [1, %d]", (long long)NB, kMaxNB);
    if (K < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "K must be >= 1");
    if (K > INT32_MAX / 2 || Hi * T > INT32_MAX / 2) return fail(SPD_ERR_UNSUPPORTED, "too many rows");
    if (!check_output_layout(o, "topk_idx")) return false;
    if (!check_no_overlap(o, "topk_idx", {s})) return false;
    if (Hi * T == 0) return true;

    SelectArgs a{};
    a.s = static_cast<const float *>(s->data); a.s_s0 = s->stride[0]; a.s_s1 = s->stride[1]; a.s_s2 = s->stride[2];
    a.o = static_cast<int32_t *>(o->data); a.o_s0 = o->stride[0]; a.o_s1 = o->stride[1]; a.o_s2 = o->stride[2];
    a.Hi = (int32_t)Hi; a.T = (int32_t)T; a.NB = (int32_t)NB; a.K = (int32_t)K;
    return check_cuda(dispatch_select(a, stream), "msa_select_topk launch");
}

// ----------------------------------------------------------------- stage 3

// What the attention calls know of their caches' scales: one static scale each,
// or one a page and kv head (block-scaled calls, E4M3 caches only).
struct Scales {
    float k = 1.f, v = 1.f;
    bool block = false;
    const spd_tensor *ks = nullptr, *vs = nullptr;
};

bool attention(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *bt,
               const spd_tensor *sl, const spd_tensor *ri, const spd_tensor *tk, const spd_tensor *out,
               float sm_scale, int32_t block_size, const Scales &sc, void *ws, size_t ws_bytes,
               cudaStream_t stream, const char *entry) {
    const spd_tensor *ks = sc.ks, *vs = sc.vs;
    if (!check_desc(q, "q", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(k, "k_cache", 3, {SPD_E4M3, SPD_BF16})) return false;
    if (!check_desc(v, "v_cache", 3, {SPD_E4M3, SPD_BF16})) return false;
    if (sc.block && (k->dtype != SPD_E4M3 || v->dtype != SPD_E4M3))
        return fail(SPD_ERR_UNSUPPORTED, "%s: block-scaled caches hold e4m3", entry);
    if (k->dtype != v->dtype) return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache and v_cache dtypes differ");
    if (!check_desc(out, "out", 3, {SPD_BF16})) return false;
    const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
    if (!check_paging(bt, sl, ri, T, block_size)) return false;
    const int64_t Hkv = k->shape[1], NB = bt->shape[1];
    for (int i = 0; i < 3; ++i)
        if (v->shape[i] != k->shape[i]) return fail(SPD_ERR_INVALID_ARGUMENT, "v_cache shape != k_cache shape");
    if (k->shape[2] != D) return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache head dim != q head dim");
    if (k->shape[0] % kBlock != 0) return fail(SPD_ERR_INVALID_ARGUMENT, "cache slots not a whole number of pages");
    if (k->stride[2] != 1 || v->stride[2] != 1)
        return fail(SPD_ERR_UNSUPPORTED, "K/V caches need a contiguous head dim");
    if (Hkv < 1 || Hq % Hkv != 0) return fail(SPD_ERR_UNSUPPORTED, "Hq=%lld not divisible by Hkv=%lld", (long long)Hq, (long long)Hkv);
    if (Hq / Hkv > kMaxGroup) return fail(SPD_ERR_UNSUPPORTED, "Hq/Hkv=%lld above %d", (long long)(Hq / Hkv), kMaxGroup);
    if (D < 1 || D > kMaxD) return fail(SPD_ERR_UNSUPPORTED, "D=%lld outside [1, %d]", (long long)D, kMaxD);
    if (Hkv > 65535 || T > INT32_MAX / 2) return fail(SPD_ERR_UNSUPPORTED, "too many heads or rows");
    if (out->shape[0] != T || out->shape[1] != Hq || out->shape[2] != D)
        return fail(SPD_ERR_INVALID_ARGUMENT, "out must be [T, Hq, D] like q");
    int64_t K = 0;
    if (tk != nullptr) {
        if (!check_desc(tk, "topk_idx", 3, {SPD_I32})) return false;
        if (tk->shape[0] != Hkv || tk->shape[1] != T)
            return fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx must be [Hkv, T, K] (stride 0 on dim 0 to share)");
        K = tk->shape[2];
        if (K < 1 || K > INT32_MAX / 2) return fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx needs K >= 1");
    }
    if (!check_scalar(sm_scale, "sm_scale") || !check_scalar(sc.k, "k_scale") || !check_scalar(sc.v, "v_scale"))
        return false;
    if (sc.block && (!check_scales(ks, "k_scales", k->shape[0] / kBlock, Hkv) ||
                     !check_scales(vs, "v_scales", k->shape[0] / kBlock, Hkv)))
        return false;
    if (!check_output_layout(out, "out")) return false;
    if (!check_no_overlap(out, "out", {q, k, v, bt, sl, ri, tk, ks, vs})) return false;
    const size_t need = spd_decode_workspace_bytes(T, Hq, Hkv, D, NB, block_size);
    if (need > 0) {
        if (ws == nullptr || ws_bytes < need)
            return fail(SPD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", entry, need, ws_bytes);
        if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
            return fail(SPD_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", entry);
        uintptr_t olo, ohi;
        byte_span(out, &olo, &ohi);
        const uintptr_t wlo = reinterpret_cast<uintptr_t>(ws), whi = wlo + ws_bytes;
        if (numel(out) > 0 && olo < whi && wlo < ohi) return fail(SPD_ERR_ALIASING, "out overlaps the workspace");
    }
    if (T == 0 || Hq == 0) return true;  // no cell to write (and no group of heads: Hq / Hkv divides below)

    AttnArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = static_cast<const uint8_t *>(k->data); a.k_s0 = k->stride[0]; a.k_s1 = k->stride[1];
    a.v = static_cast<const uint8_t *>(v->data); a.v_s0 = v->stride[0]; a.v_s1 = v->stride[1];
    a.bt = static_cast<const int32_t *>(bt->data); a.bt_s0 = bt->stride[0]; a.bt_s1 = bt->stride[1];
    a.sl = static_cast<const int32_t *>(sl->data); a.sl_s0 = sl->stride[0];
    a.ri = static_cast<const int32_t *>(ri->data); a.ri_s0 = ri->stride[0];
    if (tk != nullptr) {
        a.tk = static_cast<const int32_t *>(tk->data);
        a.tk_s0 = tk->stride[0]; a.tk_s1 = tk->stride[1]; a.tk_s2 = tk->stride[2];
    }
    a.out = static_cast<__nv_bfloat16 *>(out->data); a.o_s0 = out->stride[0]; a.o_s1 = out->stride[1]; a.o_s2 = out->stride[2];
    a.q_dt = q->dtype;
    a.kv_dt = k->dtype;
    a.T = (int32_t)T; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D;
    a.R = (int32_t)bt->shape[0]; a.NB = (int32_t)NB; a.K = (int32_t)K;
    a.P = k->shape[0] / kBlock;
    a.sm_scale = sm_scale; a.k_scale = sc.k; a.v_scale = sc.v;
    a.sc = page_scales(ks, vs);
    return check_cuda(dispatch_attention(a, ws, ws_bytes, stream), entry);
}

// ------------------------------------------- prefill score-to-selection

bool prefill_block_score(const spd_tensor *q, const spd_tensor *k, const spd_tensor *bt, const spd_tensor *sid,
                         const spd_tensor *cu_q, const spd_tensor *sl, const spd_tensor *pre, int32_t bsq,
                         int32_t bsk, int32_t init_blocks, int32_t local_blocks, float scale,
                         const spd_tensor *cu_b, const spd_tensor *out, void *ws, size_t ws_bytes,
                         cudaStream_t stream) {
    if (!check_desc(q, "q", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(k, "index_k_cache", 3, {SPD_F32, SPD_BF16, SPD_F16, SPD_E4M3})) return false;
    if (!check_desc(bt, "block_table", 2, {SPD_I32})) return false;
    if (!check_desc(sid, "slot_ids", 1, {SPD_I32})) return false;
    if (!check_desc(cu_q, "cu_seqlens", 1, {SPD_I32})) return false;
    if (!check_desc(sl, "seq_lens", 1, {SPD_I32})) return false;
    if (!check_desc(pre, "prefix_lens", 1, {SPD_I32})) return false;
    if (!check_desc(cu_b, "cu_seqblocks_q", 1, {SPD_I32})) return false;
    if (!check_desc(out, "out_topk", 3, {SPD_I32})) return false;
    const int64_t total_q = q->shape[0], Hi = q->shape[1], Di = q->shape[2];
    const int64_t B = sid->shape[0], NB = bt->shape[1];
    const int64_t n_rows = out->shape[1], topk = out->shape[2];
    if (k->dtype != q->dtype && k->dtype != SPD_E4M3)
        return fail(SPD_ERR_UNSUPPORTED, "index_k_cache dtype must match q (or be e4m3)");
    if (k->shape[1] != 1) return fail(SPD_ERR_UNSUPPORTED, "index_k_cache must have one key head");
    if (k->shape[2] != Di) return fail(SPD_ERR_INVALID_ARGUMENT, "index_k_cache head dim != q head dim");
    if (k->shape[0] % kBlock != 0) return fail(SPD_ERR_INVALID_ARGUMENT, "index_k_cache slots not a whole number of pages");
    if (sl->shape[0] != B || pre->shape[0] != B || cu_q->shape[0] != B + 1 || cu_b->shape[0] != B + 1)
        return fail(SPD_ERR_INVALID_ARGUMENT,
                    "slot_ids, seq_lens and prefix_lens need B entries, cu_seqlens and cu_seqblocks_q B + 1");
    if (bsk != kBlock) return fail(SPD_ERR_UNSUPPORTED, "block_size_k must be %d (got %d)", kBlock, bsk);
    if (bsq < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "block_size_q must be >= 1");
    if (init_blocks < 0 || local_blocks < 0) return fail(SPD_ERR_INVALID_ARGUMENT, "init/local block counts must be >= 0");
    if (!(scale > 0.f) || scale == INFINITY) return fail(SPD_ERR_UNSUPPORTED, "scale must be finite and > 0");
    if (NB < 1 || NB > kMaxNB) return fail(SPD_ERR_UNSUPPORTED, "NB=%lld outside [1, %d]", (long long)NB, kMaxNB);
    if (Di < 1 || Di > kMaxDi) return fail(SPD_ERR_UNSUPPORTED, "Di=%lld outside [1, %d]", (long long)Di, kMaxDi);
    if (Hi < 1 || Hi > 65535) return fail(SPD_ERR_UNSUPPORTED, "Hi=%lld outside [1, 65535]", (long long)Hi);
    if (out->shape[0] != Hi) return fail(SPD_ERR_INVALID_ARGUMENT, "out_topk must be [Hi, rows, topk]");
    if (topk < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "out_topk needs topk >= 1");
    if (B > INT32_MAX / 2 || total_q > INT32_MAX / 2 || n_rows > INT32_MAX / 2 || topk > INT32_MAX / 2 ||
        Hi * total_q * NB > (int64_t(1) << 40))
        return fail(SPD_ERR_UNSUPPORTED, "batch too large");
    if (B > 0 && bt->shape[0] < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "block_table has no rows");
    if (numel(out) > 0 && !check_output_layout(out, "out_topk")) return false;  // an empty output has no cells
    if (!check_no_overlap(out, "out_topk", {q, k, bt, sid, cu_q, sl, pre, cu_b})) return false;
    const size_t need = prefill_workspace_bytes(total_q, Hi, NB);
    if (need > 0 && (ws == nullptr || ws_bytes < need))
        return fail(SPD_ERR_WORKSPACE, "msa_prefill_block_score: workspace of %zu bytes needed, %zu given", need,
                    ws_bytes);
    if (need > 0 && reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return fail(SPD_ERR_WORKSPACE, "msa_prefill_block_score: workspace must be 256-byte aligned");
    if (need > 0 && numel(out) > 0) {
        uintptr_t olo, ohi;
        byte_span(out, &olo, &ohi);
        const uintptr_t wlo = reinterpret_cast<uintptr_t>(ws), whi = wlo + ws_bytes;
        if (olo < whi && wlo < ohi) return fail(SPD_ERR_ALIASING, "out_topk overlaps the workspace");
    }
    if (n_rows == 0) return true;

    PrefillArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = k->data; a.k_s0 = k->stride[0]; a.k_s2 = k->stride[2];
    a.bt = static_cast<const int32_t *>(bt->data); a.bt_s0 = bt->stride[0]; a.bt_s1 = bt->stride[1];
    a.slot_ids = static_cast<const int32_t *>(sid->data); a.sid_s0 = sid->stride[0];
    a.cu_q = static_cast<const int32_t *>(cu_q->data); a.cuq_s0 = cu_q->stride[0];
    a.seq_lens = static_cast<const int32_t *>(sl->data); a.sl_s0 = sl->stride[0];
    a.prefix = static_cast<const int32_t *>(pre->data); a.pre_s0 = pre->stride[0];
    a.cu_b = static_cast<const int32_t *>(cu_b->data); a.cub_s0 = cu_b->stride[0];
    a.out = static_cast<int32_t *>(out->data); a.o_s0 = out->stride[0]; a.o_s1 = out->stride[1]; a.o_s2 = out->stride[2];
    a.q_dt = q->dtype; a.k_dt = k->dtype;
    a.total_q = (int32_t)total_q; a.Hi = (int32_t)Hi; a.Di = (int32_t)Di; a.R = (int32_t)bt->shape[0];
    a.NB = (int32_t)NB; a.B = (int32_t)B; a.n_rows = (int32_t)n_rows; a.topk = (int32_t)topk;
    a.bsq = bsq; a.init_blocks = init_blocks; a.local_blocks = local_blocks;
    a.P = k->shape[0] / kBlock;
    a.scale = scale;
    return check_cuda(launch_prefill(a, ws, stream), "msa_prefill_block_score launch");
}

// ------------------------------------------------ slots of a serving step

// Several outputs of one call: each has a legal layout, overlaps no input and
// none of the outputs named after it.
struct Output {
    const spd_tensor *t;
    const char *name;
};

bool check_outputs(std::initializer_list<Output> outs, std::initializer_list<const spd_tensor *> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (numel(o->t) == 0) continue;
        if (!check_output_layout(o->t, o->name)) return false;
        if (!check_no_overlap(o->t, o->name, ins)) return false;
        for (auto p = o + 1; p != outs.end(); ++p) {
            if (numel(p->t) == 0) continue;
            uintptr_t alo, ahi, blo, bhi;
            byte_span(o->t, &alo, &ahi);
            byte_span(p->t, &blo, &bhi);
            if (alo < bhi && blo < ahi) return fail(SPD_ERR_ALIASING, "%s overlaps %s", o->name, p->name);
        }
    }
    return true;
}

bool assign_slots(const spd_tensor *nw, const spd_tensor *pre, const spd_tensor *sid, const spd_tensor *fp,
                  const spd_tensor *fc, int32_t n_pages, int32_t block_size, int32_t bsq, const spd_tensor *bt,
                  const spd_tensor *cu, const spd_tensor *cub, const spd_tensor *sl, const spd_tensor *req,
                  const spd_tensor *tl, const spd_tensor *slots, const spd_tensor *left, cudaStream_t stream) {
    if (!check_desc(nw, "new_lens", 1, {SPD_I32}) || !check_desc(pre, "prefix_lens", 1, {SPD_I32}) ||
        !check_desc(sid, "slot_ids", 1, {SPD_I32}) || !check_desc(fp, "free_pages", 1, {SPD_I32}) ||
        !check_desc(fc, "free_count", 1, {SPD_I32}) || !check_desc(bt, "block_table", 2, {SPD_I32}) ||
        !check_desc(cu, "cu_seqlens", 1, {SPD_I32}) || !check_desc(cub, "cu_seqblocks_q", 1, {SPD_I32}) ||
        !check_desc(sl, "seq_lens", 1, {SPD_I32}) || !check_desc(req, "req_idx", 1, {SPD_I32}) ||
        !check_desc(tl, "token_lens", 1, {SPD_I32}) || !check_desc(slots, "slots", 1, {SPD_I32}) ||
        !check_desc(left, "free_left", 1, {SPD_I32}))
        return false;
    const int64_t B = nw->shape[0], T = req->shape[0], F = fp->shape[0], NB = bt->shape[1];
    if (pre->shape[0] != B || sid->shape[0] != B || sl->shape[0] != B)
        return fail(SPD_ERR_INVALID_ARGUMENT, "prefix_lens, slot_ids and seq_lens must have B=%lld entries", (long long)B);
    if (cu->shape[0] != B + 1 || cub->shape[0] != B + 1)
        return fail(SPD_ERR_INVALID_ARGUMENT, "cu_seqlens and cu_seqblocks_q must have B + 1 entries");
    if (tl->shape[0] != T || slots->shape[0] != T)
        return fail(SPD_ERR_INVALID_ARGUMENT, "token_lens and slots must have T=%lld entries", (long long)T);
    if (fc->shape[0] != 1 || left->shape[0] != 1)
        return fail(SPD_ERR_INVALID_ARGUMENT, "free_count and free_left must have one entry");
    if (block_size != kBlock)
        return fail(SPD_ERR_UNSUPPORTED, "block_size must be %d (got %d)", kBlock, block_size);
    if (bsq < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "block_size_q must be >= 1");
    if (n_pages < 0 || n_pages > INT32_MAX / kBlock)
        return fail(SPD_ERR_UNSUPPORTED, "n_pages=%d outside [0, %d]", n_pages, INT32_MAX / kBlock);
    if (NB < 1 || NB > kMaxNB) return fail(SPD_ERR_UNSUPPORTED, "NB=%lld outside [1, %d]", (long long)NB, kMaxNB);
    if (B > kMaxSeqs) return fail(SPD_ERR_UNSUPPORTED, "B=%lld above %d", (long long)B, kMaxSeqs);
    if (T > INT32_MAX / 2 || F > INT32_MAX / 2 || bt->shape[0] > INT32_MAX / 2)
        return fail(SPD_ERR_UNSUPPORTED, "too many tokens, free pages or table rows");
    if (!check_outputs({{bt, "block_table"}, {cu, "cu_seqlens"}, {cub, "cu_seqblocks_q"}, {sl, "seq_lens"},
                        {req, "req_idx"}, {tl, "token_lens"}, {slots, "slots"}, {left, "free_left"}},
                       {nw, pre, sid, fp, fc}))
        return false;

    AssignArgs a{};
    auto in = [](const spd_tensor *t) { return static_cast<const int32_t *>(t->data); };
    auto out = [](const spd_tensor *t) { return static_cast<int32_t *>(t->data); };
    a.nw = in(nw); a.nw_s0 = nw->stride[0];
    a.pre = in(pre); a.pre_s0 = pre->stride[0];
    a.sid = in(sid); a.sid_s0 = sid->stride[0];
    a.free_pages = in(fp); a.fp_s0 = fp->stride[0];
    a.free_count = in(fc);
    a.bt = out(bt); a.bt_s0 = bt->stride[0]; a.bt_s1 = bt->stride[1];
    a.cu = out(cu); a.cu_s0 = cu->stride[0];
    a.cub = out(cub); a.cub_s0 = cub->stride[0];
    a.sl = out(sl); a.sl_s0 = sl->stride[0];
    a.req = out(req); a.req_s0 = req->stride[0];
    a.tl = out(tl); a.tl_s0 = tl->stride[0];
    a.slots = out(slots); a.slots_s0 = slots->stride[0];
    a.left = out(left);
    a.B = (int32_t)B; a.F = (int32_t)F; a.R = (int32_t)bt->shape[0]; a.NB = (int32_t)NB; a.T = (int32_t)T;
    a.n_pages = n_pages; a.bsq = bsq;
    return check_cuda(launch_assign(a, stream), "paged_assign_slots launch");
}

// ------------------------------------- norm, rotary positions, cache store

struct Dim {
    int64_t extent, stride;
};

// Whether `apart` is a distance between two cells of n dims of these extents and
// strides, the strides descending and nested: of each only two multiples can be part
// of it.
bool is_distance(const Dim *dims, int n, int64_t apart) {
    if (n == 0) return apart == 0;
    const Dim d = dims[0];
    const int64_t low = apart / d.stride - (apart % d.stride < 0 ? 1 : 0);
    for (int64_t k = low; k <= low + 1; ++k)
        if (k > -d.extent && k < d.extent && is_distance(dims + 1, n - 1, apart - k * d.stride)) return true;
    return false;
}

// Whether two outputs of one shape and legal layout whose byte spans overlap are
// still disjoint: with equal strides, as K and V beside each other in one allocation.
bool side_by_side(const spd_tensor *a, const spd_tensor *b) {
    Dim dims[4];
    int n = 0;
    for (int i = 0; i < a->ndim; ++i) {
        if (a->shape[i] <= 1) continue;
        if (a->stride[i] != b->stride[i]) return false;
        dims[n++] = {a->shape[i], a->stride[i]};
    }
    std::sort(dims, dims + n, [](const Dim &x, const Dim &y) { return x.stride > y.stride; });
    const int es = elem_size(a->dtype);
    const int64_t bytes = static_cast<int64_t>(reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data));
    return bytes % es == 0 && !is_distance(dims, n, bytes / es);
}

// K's and V's part of an output, each with a legal layout and apart from `ins` and
// from one another.
bool check_output_pair(const Output &k, const Output &v, std::initializer_list<const spd_tensor *> ins) {
    if (!check_outputs({k}, ins) || !check_outputs({v}, ins)) return false;
    if (numel(k.t) == 0 || numel(v.t) == 0) return true;
    uintptr_t alo, ahi, blo, bhi;
    byte_span(k.t, &alo, &ahi);
    byte_span(v.t, &blo, &bhi);
    if (alo < bhi && blo < ahi && !side_by_side(k.t, v.t)) return fail(SPD_ERR_ALIASING, "%s overlaps %s", k.name, v.name);
    return true;
}

bool norm_rope_store(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *wq,
                     const spd_tensor *wk, const spd_tensor *cs, const spd_tensor *tl, const spd_tensor *slots,
                     const spd_tensor *qo, const spd_tensor *kc, const spd_tensor *vc, float eps,
                     int32_t interleaved, int32_t block_size, const Scales &sc, cudaStream_t stream) {
    const spd_tensor *ks = sc.ks, *vs = sc.vs;
    if (!check_desc(q, "q", 3, {SPD_F32, SPD_BF16, SPD_F16}) || !check_desc(k, "k", 3, {SPD_F32, SPD_BF16, SPD_F16}) ||
        !check_desc(cs, "cos_sin", 2, {SPD_F32}) || !check_desc(tl, "token_lens", 1, {SPD_I32}) ||
        !check_desc(slots, "slots", 1, {SPD_I32}) || !check_desc(qo, "q_out", 3, {SPD_F32, SPD_BF16, SPD_F16}) ||
        !check_desc(kc, "k_cache", 3, {SPD_F32, SPD_BF16, SPD_F16, SPD_E4M3}))
        return false;
    if ((v == nullptr) != (vc == nullptr))
        return fail(SPD_ERR_INVALID_ARGUMENT, "v and v_cache must be given together");
    if (sc.block && v == nullptr) return fail(SPD_ERR_INVALID_ARGUMENT, "v and v_cache are needed");
    if (v != nullptr && (!check_desc(v, "v", 3, {SPD_F32, SPD_BF16, SPD_F16}) ||
                         !check_desc(vc, "v_cache", 3, {SPD_F32, SPD_BF16, SPD_F16, SPD_E4M3})))
        return false;
    const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hkv = k->shape[1];
    for (const spd_tensor *w : {wq, wk}) {
        if (w == nullptr) continue;
        const char *name = w == wq ? "q_weight" : "k_weight";
        if (!check_desc(w, name, 1, {SPD_F32, SPD_BF16, SPD_F16})) return false;
        if (w->shape[0] != D) return fail(SPD_ERR_INVALID_ARGUMENT, "%s must have D=%lld entries", name, (long long)D);
    }
    if (k->dtype != q->dtype || (v != nullptr && v->dtype != q->dtype))
        return fail(SPD_ERR_UNSUPPORTED, "k and v must have the dtype of q");
    if (vc != nullptr && vc->dtype != kc->dtype) return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache and v_cache dtypes differ");
    if (sc.block && kc->dtype != SPD_E4M3) return fail(SPD_ERR_UNSUPPORTED, "block-scaled caches hold e4m3");
    if (k->shape[0] != T || k->shape[2] != D) return fail(SPD_ERR_INVALID_ARGUMENT, "k must be [T, Hkv, D] with q's T and D");
    if (tl->shape[0] != T || slots->shape[0] != T)
        return fail(SPD_ERR_INVALID_ARGUMENT, "token_lens and slots must have T=%lld entries", (long long)T);
    if (kc->shape[1] != Hkv || kc->shape[2] != D)
        return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache must be [slots, Hkv=%lld, D=%lld]", (long long)Hkv, (long long)D);
    if (kc->shape[0] % kBlock != 0) return fail(SPD_ERR_INVALID_ARGUMENT, "cache slots not a whole number of pages");
    for (int i = 0; v != nullptr && i < 3; ++i) {
        if (v->shape[i] != k->shape[i]) return fail(SPD_ERR_INVALID_ARGUMENT, "v shape != k shape");
        if (vc->shape[i] != kc->shape[i]) return fail(SPD_ERR_INVALID_ARGUMENT, "v_cache shape != k_cache shape");
    }
    if (qo->shape[0] != T || qo->shape[1] != Hq || qo->shape[2] != D)
        return fail(SPD_ERR_INVALID_ARGUMENT, "q_out must be [T, Hq, D] like q");
    const int64_t M = cs->shape[0], Rd = cs->shape[1];
    if (block_size != kBlock) return fail(SPD_ERR_UNSUPPORTED, "block_size must be %d (got %d)", kBlock, block_size);
    if (D < 1 || D > kMaxD) return fail(SPD_ERR_UNSUPPORTED, "D=%lld outside [1, %d]", (long long)D, kMaxD);
    if (Rd < 2 || Rd > D || Rd % 2 != 0)
        return fail(SPD_ERR_UNSUPPORTED, "cos_sin must have an even number of columns in [2, D] (got %lld)", (long long)Rd);
    if (Hq < 1 || Hkv < 1 || Hq > 65535 || Hkv > 65535) return fail(SPD_ERR_UNSUPPORTED, "Hq and Hkv must be in [1, 65535]");
    if (T > INT32_MAX / 2 || M > INT32_MAX / 2 || kc->shape[0] > INT32_MAX)
        return fail(SPD_ERR_UNSUPPORTED, "too many tokens, positions or slots");
    if (!check_scalar(eps, "eps")) return false;
    if (eps < 0.f) return fail(SPD_ERR_INVALID_ARGUMENT, "eps must be >= 0");
    const float k_inv = 1.f / sc.k, v_inv = 1.f / sc.v;
    if (!(sc.k > 0.f) || !(sc.v > 0.f) || sc.k == INFINITY || sc.v == INFINITY || k_inv == INFINITY || v_inv == INFINITY)
        return fail(SPD_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be finite and > 0 with finite reciprocals");
    if (sc.block && (!check_scales(ks, "k_scales", kc->shape[0] / kBlock, Hkv) ||
                     !check_scales(vs, "v_scales", kc->shape[0] / kBlock, Hkv)))
        return false;
    if (!check_outputs({{qo, "q_out"}, {kc, "k_cache"}}, {q, k, v, wq, wk, cs, tl, slots})) return false;
    if (vc != nullptr &&
        !check_output_pair({kc, "k_cache"}, {vc, "v_cache"}, {q, k, v, wq, wk, cs, tl, slots, qo}))
        return false;
    if (sc.block &&
        !check_output_pair({ks, "k_scales"}, {vs, "v_scales"}, {q, k, v, wq, wk, cs, tl, slots, qo, kc, vc}))
        return false;
    if (T == 0) return true;

    StoreArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = k->data; a.k_s0 = k->stride[0]; a.k_s1 = k->stride[1]; a.k_s2 = k->stride[2];
    if (v != nullptr) { a.v = v->data; a.v_s0 = v->stride[0]; a.v_s1 = v->stride[1]; a.v_s2 = v->stride[2]; }
    if (wq != nullptr) { a.wq = wq->data; a.wq_s0 = wq->stride[0]; a.wq_dt = wq->dtype; }
    if (wk != nullptr) { a.wk = wk->data; a.wk_s0 = wk->stride[0]; a.wk_dt = wk->dtype; }
    a.cs = static_cast<const float *>(cs->data); a.cs_s0 = cs->stride[0]; a.cs_s1 = cs->stride[1];
    a.tl = static_cast<const int32_t *>(tl->data); a.tl_s0 = tl->stride[0];
    a.slots = static_cast<const int32_t *>(slots->data); a.slots_s0 = slots->stride[0];
    a.qo = qo->data; a.qo_s0 = qo->stride[0]; a.qo_s1 = qo->stride[1]; a.qo_s2 = qo->stride[2];
    a.kc = kc->data; a.kc_s0 = kc->stride[0]; a.kc_s1 = kc->stride[1]; a.kc_s2 = kc->stride[2];
    if (vc != nullptr) { a.vc = vc->data; a.vc_s0 = vc->stride[0]; a.vc_s1 = vc->stride[1]; a.vc_s2 = vc->stride[2]; }
    a.n_slots = kc->shape[0];
    a.in_dt = q->dtype; a.qo_dt = qo->dtype; a.c_dt = kc->dtype;
    a.T = (int32_t)T; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D; a.Rd = (int32_t)Rd; a.M = (int32_t)M;
    a.interleaved = interleaved != 0;
    a.eps = eps; a.k_inv = k_inv; a.v_inv = v_inv;
    if (sc.block) {
        a.ks = static_cast<float *>(ks->data); a.ks_s0 = ks->stride[0]; a.ks_s1 = ks->stride[1];
        a.vs = static_cast<float *>(vs->data); a.vs_s0 = vs->stride[0]; a.vs_s1 = vs->stride[1];
        return check_cuda(dispatch_store_block(a, stream), "paged_norm_rope_store_block_scaled launch");
    }
    return check_cuda(dispatch_store(a, stream), "paged_norm_rope_store launch");
}

// ------------------------------------------------------ prefill attention

bool prefill_attention(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *bt,
                       const spd_tensor *sid, const spd_tensor *cu, const spd_tensor *sl, const spd_tensor *pre,
                       const spd_tensor *tk, int32_t bsq, const spd_tensor *cub, const spd_tensor *out,
                       float sm_scale, int32_t block_size, const Scales &sc, bool sparse, void *ws,
                       size_t ws_bytes, cudaStream_t stream, const char *entry) {
    const spd_tensor *ks = sc.ks, *vs = sc.vs;
    if (!check_desc(q, "q", 3, {SPD_F32, SPD_BF16, SPD_F16}) || !check_desc(k, "k_cache", 3, {SPD_E4M3, SPD_BF16}) ||
        !check_desc(v, "v_cache", 3, {SPD_E4M3, SPD_BF16}) || !check_desc(bt, "block_table", 2, {SPD_I32}) ||
        !check_desc(sid, "slot_ids", 1, {SPD_I32}) || !check_desc(cu, "cu_seqlens", 1, {SPD_I32}) ||
        !check_desc(sl, "seq_lens", 1, {SPD_I32}) || !check_desc(pre, "prefix_lens", 1, {SPD_I32}) ||
        !check_desc(out, "out", 3, {SPD_BF16}))
        return false;
    if (sparse && (!check_desc(tk, "topk_idx", 3, {SPD_I32}) || !check_desc(cub, "cu_seqblocks_q", 1, {SPD_I32})))
        return false;
    if (sc.block && (k->dtype != SPD_E4M3 || v->dtype != SPD_E4M3))
        return fail(SPD_ERR_UNSUPPORTED, "%s: block-scaled caches hold e4m3", entry);
    if (k->dtype != v->dtype) return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache and v_cache dtypes differ");
    const int64_t total_q = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hkv = k->shape[1];
    const int64_t B = sid->shape[0], NB = bt->shape[1];
    for (int i = 0; i < 3; ++i)
        if (v->shape[i] != k->shape[i]) return fail(SPD_ERR_INVALID_ARGUMENT, "v_cache shape != k_cache shape");
    if (k->shape[2] != D) return fail(SPD_ERR_INVALID_ARGUMENT, "k_cache head dim != q head dim");
    if (k->shape[0] % kBlock != 0) return fail(SPD_ERR_INVALID_ARGUMENT, "cache slots not a whole number of pages");
    if (k->stride[2] != 1 || v->stride[2] != 1) return fail(SPD_ERR_UNSUPPORTED, "K/V caches need a contiguous head dim");
    if (sl->shape[0] != B || pre->shape[0] != B || cu->shape[0] != B + 1)
        return fail(SPD_ERR_INVALID_ARGUMENT, "seq_lens and prefix_lens need B entries, cu_seqlens B + 1");
    if (block_size != kBlock) return fail(SPD_ERR_UNSUPPORTED, "block_size must be %d (got %d)", kBlock, block_size);
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
        return fail(SPD_ERR_UNSUPPORTED, "Hq=%lld must be a positive multiple of Hkv=%lld", (long long)Hq, (long long)Hkv);
    if (Hq / Hkv > kMaxGroup) return fail(SPD_ERR_UNSUPPORTED, "Hq/Hkv=%lld above %d", (long long)(Hq / Hkv), kMaxGroup);
    if (D < 1 || D > kMaxD) return fail(SPD_ERR_UNSUPPORTED, "D=%lld outside [1, %d]", (long long)D, kMaxD);
    if (NB < 1 || NB > kMaxNB) return fail(SPD_ERR_UNSUPPORTED, "NB=%lld outside [1, %d]", (long long)NB, kMaxNB);
    if (B > kMaxSeqs) return fail(SPD_ERR_UNSUPPORTED, "B=%lld above %d", (long long)B, kMaxSeqs);
    if (Hkv > 65535 || total_q > INT32_MAX / 2 || total_q * Hq > INT32_MAX / 2 || bt->shape[0] > INT32_MAX / 2 ||
        k->shape[0] > INT32_MAX)
        return fail(SPD_ERR_UNSUPPORTED, "too many heads, query rows, table rows or slots");
    int64_t n_rows = 0, K = 0;
    if (sparse) {
        n_rows = tk->shape[1];
        K = tk->shape[2];
        if (tk->shape[0] != Hkv)
            return fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx must be [Hkv, rows, K] (stride 0 on dim 0 to share)");
        if (cub->shape[0] != B + 1) return fail(SPD_ERR_INVALID_ARGUMENT, "cu_seqblocks_q needs B + 1 entries");
        if (K < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx needs K >= 1");
        if (K > INT32_MAX / 2 || n_rows > INT32_MAX / 2) return fail(SPD_ERR_UNSUPPORTED, "topk_idx too large");
        if (bsq < 1) return fail(SPD_ERR_INVALID_ARGUMENT, "block_size_q must be >= 1");
    }
    if (out->shape[0] != total_q || out->shape[1] != Hq || out->shape[2] != D)
        return fail(SPD_ERR_INVALID_ARGUMENT, "out must be [total_q, Hq, D] like q");
    if (!check_scalar(sm_scale, "sm_scale") || !check_scalar(sc.k, "k_scale") || !check_scalar(sc.v, "v_scale"))
        return false;
    if (sc.block && (!check_scales(ks, "k_scales", k->shape[0] / kBlock, Hkv) ||
                     !check_scales(vs, "v_scales", k->shape[0] / kBlock, Hkv)))
        return false;
    if (!check_outputs({{out, "out"}}, {q, k, v, bt, sid, cu, sl, pre, tk, cub, ks, vs})) return false;
    const size_t need = spd_prefill_attention_workspace_bytes(total_q, Hq, Hkv, D, B, NB, n_rows);
    if (ws == nullptr || ws_bytes < need)
        return fail(SPD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", entry, need, ws_bytes);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return fail(SPD_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", entry);
    const uintptr_t wlo = reinterpret_cast<uintptr_t>(ws), whi = wlo + ws_bytes;
    for (const spd_tensor *t : {out, q, k, v, bt, sid, cu, sl, pre, tk, cub, ks, vs}) {
        if (t == nullptr || numel(t) == 0) continue;
        uintptr_t lo, hi;
        byte_span(t, &lo, &hi);
        if (lo < whi && wlo < hi) return fail(SPD_ERR_ALIASING, "%s: a tensor overlaps the workspace", entry);
    }
    if (total_q == 0) return true;

    ChunkArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = static_cast<const uint8_t *>(k->data); a.k_s0 = k->stride[0]; a.k_s1 = k->stride[1];
    a.v = static_cast<const uint8_t *>(v->data); a.v_s0 = v->stride[0]; a.v_s1 = v->stride[1];
    a.bt = static_cast<const int32_t *>(bt->data); a.bt_s0 = bt->stride[0]; a.bt_s1 = bt->stride[1];
    a.sid = static_cast<const int32_t *>(sid->data); a.sid_s0 = sid->stride[0];
    a.cu = static_cast<const int32_t *>(cu->data); a.cu_s0 = cu->stride[0];
    a.sl = static_cast<const int32_t *>(sl->data); a.sl_s0 = sl->stride[0];
    a.pre = static_cast<const int32_t *>(pre->data); a.pre_s0 = pre->stride[0];
    if (sparse) {
        // an address says that there is a selection; of one without rows
        // nothing is read, and its tensor has none
        a.tk = static_cast<const int32_t *>(n_rows > 0 ? tk->data : cu->data);
        a.tk_s0 = tk->stride[0]; a.tk_s1 = tk->stride[1]; a.tk_s2 = tk->stride[2];
        a.cub = static_cast<const int32_t *>(cub->data); a.cub_s0 = cub->stride[0];
        a.n_rows = (int32_t)n_rows; a.K = (int32_t)K; a.bsq = bsq;
    }
    a.out = out->data; a.o_s0 = out->stride[0]; a.o_s1 = out->stride[1]; a.o_s2 = out->stride[2];
    a.q_dt = q->dtype; a.kv_dt = k->dtype;
    a.total_q = (int32_t)total_q; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D;
    a.B = (int32_t)B; a.R = (int32_t)bt->shape[0]; a.NB = (int32_t)NB;
    a.P = k->shape[0] / kBlock;
    a.sm_scale = sm_scale; a.k_scale = sc.k; a.v_scale = sc.v;
    a.sc = page_scales(ks, vs);
    return check_cuda(dispatch_chunk(a, ws, ws_bytes, stream), entry);
}

// ------------------------------------------------------- dense attention

bool sdpa(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *out, float sm_scale,
          int32_t causal, cudaStream_t stream) {
    if (!check_desc(q, "q", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(k, "k", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(v, "v", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (!check_desc(out, "out", 3, {SPD_F32, SPD_BF16, SPD_F16})) return false;
    if (k->dtype != q->dtype || v->dtype != q->dtype)
        return fail(SPD_ERR_UNSUPPORTED, "k and v must have the dtype of q");
    const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
    const int64_t S = k->shape[0], Hkv = k->shape[1];
    for (int i = 0; i < 3; ++i)
        if (v->shape[i] != k->shape[i]) return fail(SPD_ERR_INVALID_ARGUMENT, "v shape != k shape");
    if (k->shape[2] != D) return fail(SPD_ERR_INVALID_ARGUMENT, "k head dim != q head dim");
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
        return fail(SPD_ERR_UNSUPPORTED, "Hq=%lld must be a positive multiple of Hkv=%lld", (long long)Hq,
                    (long long)Hkv);
    if (D < 1 || D > kMaxD) return fail(SPD_ERR_UNSUPPORTED, "D=%lld outside [1, %d]", (long long)D, kMaxD);
    if (Hkv > 65535 || S > INT32_MAX / 2 || T > INT32_MAX / 2 || T * Hq > INT32_MAX / 2)
        return fail(SPD_ERR_UNSUPPORTED, "too many heads, keys or query rows");
    if (out->shape[0] != T || out->shape[1] != Hq || out->shape[2] != D)
        return fail(SPD_ERR_INVALID_ARGUMENT, "out must be [T, Hq, D] like q");
    if (!check_scalar(sm_scale, "sm_scale")) return false;
    if (!check_output_layout(out, "out")) return false;
    if (!check_no_overlap(out, "out", {q, k, v})) return false;
    if (T == 0) return true;

    SdpaArgs a{};
    a.q = q->data; a.q_s0 = q->stride[0]; a.q_s1 = q->stride[1]; a.q_s2 = q->stride[2];
    a.k = k->data; a.k_s0 = k->stride[0]; a.k_s1 = k->stride[1]; a.k_s2 = k->stride[2];
    a.v = v->data; a.v_s0 = v->stride[0]; a.v_s1 = v->stride[1]; a.v_s2 = v->stride[2];
    a.out = out->data; a.o_s0 = out->stride[0]; a.o_s1 = out->stride[1]; a.o_s2 = out->stride[2];
    a.in_dt = q->dtype; a.out_dt = out->dtype;
    a.T = (int32_t)T; a.S = (int32_t)S; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D;
    a.causal = causal != 0;
    a.sm_scale = sm_scale;
    return check_cuda(dispatch_sdpa(a, stream), "attention_sdpa launch");
}

}  // namespace
}  // namespace spd

// ============================================ attention with built-in scratch
//
// Scratch for paged_sparse_decode_attention_noalloc: a fixed device array
// that belongs to the library, so the caller never has to provide (or
// allocate) a workspace.  It is created with the library's device code on each
// GPU where the entry point is used and stays until the process exits.
static constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

namespace spd {
namespace {

std::mutex g_noalloc_mu;
void *g_noalloc_ptr[256] = {};

// Device address of g_noalloc_scratch on the current device.  The name is
// only a host-side stand-in for the array, so the address is looked up with
// cudaGetSymbolAddress, once per device and with that device current.
void *noalloc_scratch() {
    int dev = 0;
    if (!check_cuda(cudaGetDevice(&dev), "paged_sparse_decode_attention_noalloc: cudaGetDevice")) return nullptr;
    if (dev < 0 || dev >= 256) {
        fail(SPD_ERR_UNSUPPORTED, "paged_sparse_decode_attention_noalloc: device ordinal %d out of range", dev);
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    if (g_noalloc_ptr[dev] == nullptr) {
        void *p = nullptr;
        if (!check_cuda(cudaGetSymbolAddress(&p, g_noalloc_scratch),
                        "paged_sparse_decode_attention_noalloc: cudaGetSymbolAddress"))
            return nullptr;
        g_noalloc_ptr[dev] = p;
    }
    return g_noalloc_ptr[dev];
}

}  // namespace
}  // namespace spd

// ======================================================================= ABI

extern "C" {

void msa_block_score(const spd_tensor *q_idx, const spd_tensor *k_idx_cache, const spd_tensor *block_table,
                     const spd_tensor *seq_lens, const spd_tensor *req_idx, int32_t block_size,
                     const spd_tensor *scores, float idx_scale, spd_stream_t stream) {
    spd::set_ok();
    spd::block_score(q_idx, k_idx_cache, block_table, seq_lens, req_idx, block_size, scores, idx_scale,
                     reinterpret_cast<cudaStream_t>(stream));
}

void msa_select_topk(const spd_tensor *scores, const spd_tensor *topk_idx, spd_stream_t stream) {
    spd::set_ok();
    spd::select_topk(scores, topk_idx, reinterpret_cast<cudaStream_t>(stream));
}

void paged_sparse_decode_attention(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                                   const spd_tensor *block_table, const spd_tensor *seq_lens,
                                   const spd_tensor *req_idx, const spd_tensor *topk_idx, const spd_tensor *out,
                                   float sm_scale, int32_t block_size, float k_scale, float v_scale,
                                   void *workspace, size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    if (topk_idx == nullptr) {
        spd::fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx is NULL (use paged_decode_attention for dense decode)");
        return;
    }
    spd::attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, topk_idx, out, sm_scale, block_size,
                   {k_scale, v_scale}, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream),
                   "paged_sparse_decode_attention");
}

void paged_sparse_decode_attention_noalloc(const spd_tensor *q, const spd_tensor *k_cache,
                                           const spd_tensor *v_cache, const spd_tensor *block_table,
                                           const spd_tensor *seq_lens, const spd_tensor *req_idx,
                                           const spd_tensor *topk_idx, const spd_tensor *out, float sm_scale,
                                           int32_t block_size, float k_scale, float v_scale, spd_stream_t stream) {
    spd::set_ok();
    if (topk_idx == nullptr) {
        spd::fail(SPD_ERR_INVALID_ARGUMENT, "topk_idx is NULL");
        return;
    }
    if (q != nullptr && k_cache != nullptr && block_table != nullptr && q->ndim == 3 && k_cache->ndim == 3 &&
        block_table->ndim == 2) {
        const size_t need = spd_decode_workspace_bytes(q->shape[0], q->shape[1], k_cache->shape[1], q->shape[2],
                                                       block_table->shape[1], block_size);
        if (need > kNoAllocScratchBytes) {
            spd::fail(SPD_ERR_UNSUPPORTED,
                      "paged_sparse_decode_attention_noalloc: this shape needs %zu bytes of scratch, more than the "
                      "%zu-byte scratch built into the library; use paged_sparse_decode_attention with a workspace",
                      need, kNoAllocScratchBytes);
            return;
        }
    }
    void *ws = spd::noalloc_scratch();
    if (ws == nullptr) return;
    // everything the kernels need to start from zero (the per-pair merge
    // counters, the status word) is written by this call's planner kernel
    spd::attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, topk_idx, out, sm_scale, block_size,
                   {k_scale, v_scale}, ws, kNoAllocScratchBytes, reinterpret_cast<cudaStream_t>(stream),
                   "paged_sparse_decode_attention_noalloc");
}

void paged_decode_attention(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                            const spd_tensor *block_table, const spd_tensor *seq_lens, const spd_tensor *req_idx,
                            const spd_tensor *out, float sm_scale, int32_t block_size, float k_scale,
                            float v_scale, void *workspace, size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    spd::attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, nullptr, out, sm_scale, block_size,
                   {k_scale, v_scale}, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream),
                   "paged_decode_attention");
}

void msa_prefill_block_score(const spd_tensor *q, const spd_tensor *index_k_cache, const spd_tensor *block_table,
                             const spd_tensor *slot_ids, const spd_tensor *cu_seqlens, const spd_tensor *seq_lens,
                             const spd_tensor *prefix_lens, int32_t block_size_q, int32_t block_size_k,
                             int32_t init_blocks, int32_t local_blocks, float scale,
                             const spd_tensor *cu_seqblocks_q, const spd_tensor *out_topk, void *workspace,
                             size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    spd::prefill_block_score(q, index_k_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens,
                             block_size_q, block_size_k, init_blocks, local_blocks, scale, cu_seqblocks_q, out_topk,
                             workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t spd_prefill_workspace_bytes(int64_t total_q, int64_t Hi, int64_t NB) {
    if (total_q < 0 || Hi < 1 || NB < 1) return 0;
    return spd::prefill_workspace_bytes(total_q, Hi, NB);
}

void attention_sdpa(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *out,
                    float sm_scale, int32_t causal, spd_stream_t stream) {
    spd::set_ok();
    spd::sdpa(q, k, v, out, sm_scale, causal, reinterpret_cast<cudaStream_t>(stream));
}

void paged_assign_slots(const spd_tensor *new_lens, const spd_tensor *prefix_lens, const spd_tensor *slot_ids,
                        const spd_tensor *free_pages, const spd_tensor *free_count, int32_t n_pages,
                        int32_t block_size, int32_t block_size_q, const spd_tensor *block_table,
                        const spd_tensor *cu_seqlens, const spd_tensor *cu_seqblocks_q, const spd_tensor *seq_lens,
                        const spd_tensor *req_idx, const spd_tensor *token_lens, const spd_tensor *slots,
                        const spd_tensor *free_left, spd_stream_t stream) {
    spd::set_ok();
    spd::assign_slots(new_lens, prefix_lens, slot_ids, free_pages, free_count, n_pages, block_size, block_size_q,
                      block_table, cu_seqlens, cu_seqblocks_q, seq_lens, req_idx, token_lens, slots, free_left,
                      reinterpret_cast<cudaStream_t>(stream));
}

void paged_norm_rope_store(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v, const spd_tensor *q_weight,
                           const spd_tensor *k_weight, const spd_tensor *cos_sin, const spd_tensor *token_lens,
                           const spd_tensor *slots, const spd_tensor *q_out, const spd_tensor *k_cache,
                           const spd_tensor *v_cache, float eps, int32_t interleaved, int32_t block_size,
                           float k_scale, float v_scale, spd_stream_t stream) {
    spd::set_ok();
    spd::norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache, v_cache, eps,
                         interleaved, block_size, {k_scale, v_scale}, reinterpret_cast<cudaStream_t>(stream));
}

void paged_prefill_attention(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                             const spd_tensor *block_table, const spd_tensor *slot_ids, const spd_tensor *cu_seqlens,
                             const spd_tensor *seq_lens, const spd_tensor *prefix_lens, const spd_tensor *out,
                             float sm_scale, int32_t block_size, float k_scale, float v_scale, void *workspace,
                             size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    spd::prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens, nullptr, 1,
                           nullptr, out, sm_scale, block_size, {k_scale, v_scale}, false, workspace, workspace_bytes,
                           reinterpret_cast<cudaStream_t>(stream), "paged_prefill_attention");
}

void paged_sparse_prefill_attention(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                                    const spd_tensor *block_table, const spd_tensor *slot_ids,
                                    const spd_tensor *cu_seqlens, const spd_tensor *seq_lens,
                                    const spd_tensor *prefix_lens, const spd_tensor *topk_idx, int32_t block_size_q,
                                    const spd_tensor *cu_seqblocks_q, const spd_tensor *out, float sm_scale,
                                    int32_t block_size, float k_scale, float v_scale, void *workspace,
                                    size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    spd::prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens, topk_idx,
                           block_size_q, cu_seqblocks_q, out, sm_scale, block_size, {k_scale, v_scale}, true, workspace,
                           workspace_bytes, reinterpret_cast<cudaStream_t>(stream), "paged_sparse_prefill_attention");
}

void paged_norm_rope_store_block_scaled(const spd_tensor *q, const spd_tensor *k, const spd_tensor *v,
                                        const spd_tensor *q_weight, const spd_tensor *k_weight,
                                        const spd_tensor *cos_sin, const spd_tensor *token_lens,
                                        const spd_tensor *slots, const spd_tensor *q_out, const spd_tensor *k_cache,
                                        const spd_tensor *v_cache, const spd_tensor *k_scales,
                                        const spd_tensor *v_scales, float eps, int32_t interleaved,
                                        int32_t block_size, spd_stream_t stream) {
    spd::set_ok();
    spd::norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache, v_cache, eps,
                         interleaved, block_size, {1.f, 1.f, true, k_scales, v_scales},
                         reinterpret_cast<cudaStream_t>(stream));
}

void paged_decode_attention_block_scaled(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                                         const spd_tensor *k_scales, const spd_tensor *v_scales,
                                         const spd_tensor *block_table, const spd_tensor *seq_lens,
                                         const spd_tensor *req_idx, const spd_tensor *out, float sm_scale,
                                         int32_t block_size, void *workspace, size_t workspace_bytes,
                                         spd_stream_t stream) {
    spd::set_ok();
    spd::attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, nullptr, out, sm_scale, block_size,
                   {1.f, 1.f, true, k_scales, v_scales}, workspace, workspace_bytes,
                   reinterpret_cast<cudaStream_t>(stream), "paged_decode_attention_block_scaled");
}

void paged_sparse_decode_attention_block_scaled(const spd_tensor *q, const spd_tensor *k_cache,
                                                const spd_tensor *v_cache, const spd_tensor *k_scales,
                                                const spd_tensor *v_scales, const spd_tensor *block_table,
                                                const spd_tensor *seq_lens, const spd_tensor *req_idx,
                                                const spd_tensor *topk_idx, const spd_tensor *out, float sm_scale,
                                                int32_t block_size, void *workspace, size_t workspace_bytes,
                                                spd_stream_t stream) {
    spd::set_ok();
    if (topk_idx == nullptr) {
        spd::fail(SPD_ERR_INVALID_ARGUMENT,
                  "topk_idx is NULL (use paged_decode_attention_block_scaled for dense decode)");
        return;
    }
    spd::attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, topk_idx, out, sm_scale, block_size,
                   {1.f, 1.f, true, k_scales, v_scales}, workspace, workspace_bytes,
                   reinterpret_cast<cudaStream_t>(stream), "paged_sparse_decode_attention_block_scaled");
}

void paged_prefill_attention_block_scaled(const spd_tensor *q, const spd_tensor *k_cache, const spd_tensor *v_cache,
                                          const spd_tensor *k_scales, const spd_tensor *v_scales,
                                          const spd_tensor *block_table, const spd_tensor *slot_ids,
                                          const spd_tensor *cu_seqlens, const spd_tensor *seq_lens,
                                          const spd_tensor *prefix_lens, const spd_tensor *out, float sm_scale,
                                          int32_t block_size, void *workspace, size_t workspace_bytes,
                                          spd_stream_t stream) {
    spd::set_ok();
    spd::prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens, nullptr, 1,
                           nullptr, out, sm_scale, block_size, {1.f, 1.f, true, k_scales, v_scales}, false, workspace,
                           workspace_bytes, reinterpret_cast<cudaStream_t>(stream),
                           "paged_prefill_attention_block_scaled");
}

void paged_sparse_prefill_attention_block_scaled(const spd_tensor *q, const spd_tensor *k_cache,
                                                 const spd_tensor *v_cache, const spd_tensor *k_scales,
                                                 const spd_tensor *v_scales, const spd_tensor *block_table,
                                                 const spd_tensor *slot_ids, const spd_tensor *cu_seqlens,
                                                 const spd_tensor *seq_lens, const spd_tensor *prefix_lens,
                                                 const spd_tensor *topk_idx, int32_t block_size_q,
                                                 const spd_tensor *cu_seqblocks_q, const spd_tensor *out,
                                                 float sm_scale, int32_t block_size, void *workspace,
                                                 size_t workspace_bytes, spd_stream_t stream) {
    spd::set_ok();
    spd::prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens, topk_idx,
                           block_size_q, cu_seqblocks_q, out, sm_scale, block_size,
                           {1.f, 1.f, true, k_scales, v_scales}, true, workspace, workspace_bytes,
                           reinterpret_cast<cudaStream_t>(stream), "paged_sparse_prefill_attention_block_scaled");
}

size_t spd_prefill_attention_workspace_bytes(int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t B,
                                             int64_t NB, int64_t n_rows) {
    if (total_q < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > spd::kMaxGroup || Hkv > 65535 || D < 1 ||
        D > spd::kMaxD || B < 0 || B > spd::kMaxSeqs || NB < 1 || NB > spd::kMaxNB || n_rows < 0 ||
        n_rows > INT32_MAX / 2 || total_q > INT32_MAX / 2 || total_q * Hq > INT32_MAX / 2)
        return 0;
    return spd::chunk_workspace_bytes(total_q, Hq, Hkv, D, B, NB, n_rows);
}

size_t spd_decode_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t NB, int32_t block_size) {
    if (T < 0 || Hq < 1 || Hkv < 1 || D < 1 || NB < 1 || block_size != spd::kBlock) return 0;
    return spd::workspace_bytes(T, Hq, Hkv, D, NB);
}

int spd_last_error(char *msg, size_t cap) {
    if (msg != nullptr && cap > 0) {
        strncpy(msg, spd::g_msg, cap - 1);
        msg[cap - 1] = '\0';
    }
    return spd::g_status;
}

uint64_t spd_launch_count(void) { return spd::launch_count(); }

int spd_set_attention_kernel(int policy) { return spd::set_kernel_policy(3, policy); }

int spd_set_kernel_policy(int stage, int policy) {
    return stage >= 5 ? spd::set_serve_policy(stage, policy) : spd::set_kernel_policy(stage, policy);
}

int spd_workspace_status(const void *workspace, spd_stream_t stream) {
    if (workspace == nullptr) {
        // the built-in scratch of paged_sparse_decode_attention_noalloc on the
        // current device (a device array is zero when no call has used it)
        const int saved = spd::g_status;
        char saved_msg[sizeof spd::g_msg];
        memcpy(saved_msg, spd::g_msg, sizeof saved_msg);
        workspace = spd::noalloc_scratch();
        spd::g_status = saved;  // a diagnostic leaves the last call's status alone
        memcpy(spd::g_msg, saved_msg, sizeof saved_msg);
        if (workspace == nullptr) return -1;
    }
    return spd::workspace_status(workspace, reinterpret_cast<cudaStream_t>(stream));
}

const char *spd_version(void) { return "spd 0.1 sm_103a"; }

}  // extern "C"
