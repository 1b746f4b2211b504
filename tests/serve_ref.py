"""Plain 64-bit definitions of the serving-step calls (paged_assign_slots,
paged_norm_rope_store, paged_prefill_attention and its sparse form), written
from the formulas in include/spd.h with loops over requests, tokens and heads.

Tolerances (derived here, applied by every test of these calls).  u(t) is the
largest relative error of one rounding to type t, finfo(t).eps / 2: bf16 2^-8,
f16 2^-11, f32 2^-24, e4m3 2^-4.
  * paged_assign_slots: whole numbers, equal.
  * paged_norm_rope_store: the fp32 value carries the error of a sum of D <=
    256 squares (pairwise over 32 lanes: at most 8 + 5 roundings), a
    reciprocal root (2 ulp), two or three products, and of the rotation, whose
    two terms may cancel: at most 32 u(f32) of |a| + |b| in all.  The kept
    value is rounded once: u(t) |ref|, or half of E4M3's smallest step (2^-10)
    below its normal range.
  * prefill attention: p = exp(z - m) is rounded to bf16 (or f16) before the
    product with V: u(bf16) * A with A = sum p |v| / sum p; the logits' fp32
    error (128 products, |z| of a few tens) and the sums' together stay below
    2^-10 A; the output is rounded to bf16: u(bf16) |ref|.  So
    |got - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) A.
"""
import numpy as np
import torch

BS = 128
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
STEP = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t is not None else None


def ints(t):
    return t.detach().cpu().numpy().astype(np.int64)


def assign(new, prefix, rows, free, count, n_pages, bq, table, T):
    """(table, cu, cu_blocks, seq_lens, req, lens, slots, left) of the call."""
    new, prefix, rows, free = (ints(x) for x in (new, prefix, rows, free))
    table = ints(table).copy()
    count = max(0, min(int(count), len(free)))
    R, NB = table.shape
    B, cap = len(new), NB * BS
    cu, cub, sl = [0], [0], []
    req, lens, slots = np.full(T, -1), np.zeros(T, np.int64), np.full(T, -1)
    used = 0
    for b in range(B):
        n = min(max(int(new[b]), 0), T - cu[-1])
        p = max(int(prefix[b]), 0)
        cu.append(cu[-1] + n)
        cub.append(cub[-1] + -(-n // bq))
        sl.append(min(p + n, 2 ** 31 - 1))
        inside = 0 <= rows[b] < R
        if inside:
            for blk in range(-(-min(p, cap) // BS), -(-min(p + n, cap) // BS)):
                table[rows[b], blk] = free[count - 1 - used] if used < count else -1
                used += 1
        for i in range(n):
            t, pos = cu[b] + i, p + i
            req[t], lens[t] = rows[b], min(pos + 1, 2 ** 31 - 1)
            if inside and pos < cap and 0 <= table[rows[b], pos // BS] < n_pages:
                slots[t] = table[rows[b], pos // BS] * BS + pos % BS
    return table, np.array(cu), np.array(cub), np.array(sl, np.int64), req, lens, slots, np.array([max(0, count - used)])


def head_rows(x, w, cos_sin, lens, eps, interleaved):
    """Normalised and rotated rows of x [T, H, D] in 64 bits, and the |a| + |b| of each cell's rotation."""
    x, cs = f64(x).copy(), f64(cos_sin)
    T, H, D = x.shape
    half = cs.shape[1] // 2
    mag = np.abs(x)
    for t in range(T):
        if not 1 <= lens[t] <= cs.shape[0]:
            x[t], mag[t] = 0.0, 0.0
            continue
        for h in range(H):
            y = x[t, h]
            if w is not None:
                y = y * f64(w) / np.sqrt(np.mean(y * y) + eps)
            co, si = cs[lens[t] - 1, :half], cs[lens[t] - 1, half:]
            a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
            out, m = y.copy(), np.abs(y)
            out[a], out[b] = y[a] * co - y[b] * si, y[b] * co + y[a] * si
            m[a] = m[b] = np.abs(y[a]) + np.abs(y[b])
            x[t, h], mag[t, h] = out, m
    return x, mag


def check_kept(got, ref, mag, dtype, what):
    """Cells kept in `dtype` against their 64-bit values (already divided by the scale)."""
    got = f64(got)
    if dtype == torch.float8_e4m3fn:
        ref = np.clip(ref, -448.0, 448.0)
    tol = U[dtype] * np.abs(ref) + STEP[dtype] + 32 * U[torch.float32] * mag
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what + ": NaN pattern"
    bad = np.abs(got - ref) > tol
    assert not bad.any(), "%s: %d cells off, worst %.3g over its bound" % (what, bad.sum(), np.nanmax(np.abs(got - ref) - tol))


def readable(table, row, pool, limit, chosen=None):
    """Slots of the keys below `limit` of table row `row`, of the chosen blocks only when given."""
    if not 0 <= row < table.shape[0]:
        return np.zeros(0, np.int64)
    limit = min(limit, table.shape[1] * BS)
    out = []
    for kb in range(-(-limit // BS) if limit > 0 else 0):
        page = table[row, kb]
        if not 0 <= page < pool or (chosen is not None and kb not in chosen):
            continue
        out.append(page * BS + np.arange(min(BS, limit - kb * BS)))
    return np.concatenate(out) if out else np.zeros(0, np.int64)


def attention(q, k_cache, v_cache, table, rows, cu, seq_lens, prefix, sm_scale, k_scale, v_scale, topk=None, bq=1, cub=None):
    """(out, A) of the prefill attention calls."""
    q, kc, vc = f64(q), f64(k_cache), f64(v_cache)
    table, rows, cu, seq_lens, prefix = (ints(x) for x in (table, rows, cu, seq_lens, prefix))
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    if topk is not None:
        topk, cub = ints(topk), ints(cub)
    out, A = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(rows)):
        for t in range(cu[b], cu[b + 1]):
            i = t - cu[b]
            limit = min(prefix[b] + i + 1, seq_lens[b])
            for h in range(Hkv):
                chosen = None
                if topk is not None:
                    r = cub[b] + i // bq
                    chosen = set(topk[h, r].tolist()) if r < min(cub[b + 1], topk.shape[1]) else set()
                s = readable(table, rows[b], kc.shape[0] // BS, limit, chosen)
                if not len(s):
                    continue
                z = (q[t, h * G:(h + 1) * G] @ (kc[s, h] * k_scale).T) * sm_scale
                p = np.exp(z - z.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[t, h * G:(h + 1) * G] = p @ (vc[s, h] * v_scale)
                A[t, h * G:(h + 1) * G] = p @ (np.abs(vc[s, h]) * v_scale)
    return out, A


def check_attention(got, ref, A, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), "%s: %d cells not finite" % (what, (~np.isfinite(got)).sum())
    over = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * A)
    assert (over <= 0).all(), "%s: %d cells off, worst %.3g over its bound (token %d)" % (
        what, (over > 0).sum(), over.max(), np.unravel_index(over.argmax(), over.shape)[0])
    assert not got[A == 0].any(), what + ": a row that reads nothing is not zero"
