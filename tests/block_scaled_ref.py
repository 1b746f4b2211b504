"""Plain 64-bit definitions of the block-scaled calls, on top of serve_ref.py.

Tolerances (derived here, applied by every test of these calls; u(t) as in
serve_ref.py):
  * store: q_out and codes as paged_norm_rope_store's, the codes against y / scale.
    A scale that is written is the smallest 2^e, e in [-64, 64], that brings the run's
    largest magnitude to 448; that one is known to 32 u(f32) of the |a| + |b| of
    its cell, so either of two neighbouring powers passes where it lies within
    that of 448 2^e, and no other.  A held code is a product of a code and a
    ratio (exact in fp32 for powers of two, else off by u(f32)), rounded once.
  * attention: serve_ref's bound over the dequantised caches.  The weights
    that are rounded to f16 are p vs / w, w the row's largest such product (at a
    raise of its offset; the products may exceed it, never be below it): below 2^-14 a rounding
    is off by at most 2^-25 w, so a key adds at most 2^-25 w 448 to the bound (the kernel of
    single rows is granted 2^-22 by the header; here it has to do with this).  A scale
    enters by its logarithm, whose error of 2^-22 (and the fp32 sum's with an
    offset of up to a few hundred, 2^-16) moves a weight by less than 2^-15 of
    itself: inside the 2^-10 A that serve_ref grants to logits, next to whose 2^-11 it stays.
"""
import numpy as np
import torch

import serve_ref as R

BS = R.BS
LEAST, MOST = -64, 64


def runs(lens, slots, M, n_slots):
    """[(first row, rows, page, offset)] of the stored rows of a batch, in any order of pages."""
    lens, slots = R.ints(lens), R.ints(slots)
    out = []
    for t, (n, s) in enumerate(zip(lens, slots)):
        if not (1 <= n <= M and 0 <= s < n_slots):
            continue
        if out:
            first, rows, page, offset = out[-1]
            if first + rows == t and page * BS + offset + rows == s and offset + rows < BS:
                out[-1] = (first, rows + 1, page, offset)
                continue
        out.append((t, 1, s // BS, s % BS))
    return out


def check_store(s, before, after, q_out, eps, interleaved, what):
    """`s`: q, k, v, wq, wk, cos_sin, lens, slots; `before` and `after`: kc, vc, ks, vs as float64 arrays."""
    M = s["cos_sin"].shape[0]
    lens = R.ints(s["lens"])
    q, mag = R.head_rows(s["q"], s["wq"], s["cos_sin"], lens, eps, interleaved)
    R.check_kept(q_out, q, mag, q_out.dtype, what + ": q_out")
    k, kmag = R.head_rows(s["k"], s["wk"], s["cos_sin"], lens, eps, interleaved)
    v = R.f64(s["v"])
    parts = runs(s["lens"], s["slots"], M, before["kc"].shape[0])
    for name, y, mag in (("k", k, kmag), ("v", v, np.zeros_like(v))):
        codes, scales = before[name + "c"].copy(), before[name + "s"].copy()
        got_codes, got_scales = after[name + "c"], after[name + "s"]
        tol = np.zeros_like(codes)
        for first, rows, page, offset in parts:
            for h in range(y.shape[1]):
                new, m = y[first:first + rows, h], mag[first:first + rows, h]
                err = 32 * R.U[torch.float32] * (m.max() if np.isfinite(m).all() else 0.0)
                fin = np.abs(new[np.isfinite(new)])
                top = fin.max() if fin.size else 0.0

                def power(x):
                    if not x > 0:
                        return 2.0 ** LEAST
                    frac, e = np.frexp(x / 448.0)
                    return 2.0 ** min(MOST, max(LEAST, e - 1 if frac == 0.5 else e))

                old = scales[page, h] if offset > 0 else 0.0
                old = old if np.isfinite(old) and old > 0 else 0.0
                allowed = {old if old >= p else p for p in (power(top - err), power(top + err))}
                scale = got_scales[page, h]
                assert scale in allowed, "%s: %s scale of page %d head %d is %g, not of %r" % (what, name, page, h, scale, allowed)
                scales[page, h] = scale
                at = page * BS + offset
                codes[at:at + rows, h] = new / scale
                tol[at:at + rows, h] = m / scale + (0.0 if scale == 2.0 ** np.round(np.log2(scale)) else np.nan_to_num(np.abs(new), posinf=0.0) / scale / 8)
                if old and scale != old:
                    held = codes[page * BS:at, h] * (old / scale)
                    codes[page * BS:at, h] = held
                    tol[page * BS:at, h] = np.abs(np.nan_to_num(held)) / 8
        assert np.array_equal(got_scales, scales, equal_nan=True), "%s: %s scales of other pages changed" % (what, name)
        same = np.ones(codes.shape[0], bool)  # slots that no run or growth touches: bit for bit
        for _, rows, page, offset in parts:
            same[page * BS:page * BS + offset + rows] = False
        assert np.array_equal(got_codes[same], before[name + "c"][same], equal_nan=True), "%s: %s slots outside the runs changed" % (what, name)
        R.check_kept(torch.from_numpy(got_codes), codes, tol, torch.float8_e4m3fn, "%s: %s codes" % (what, name))


def kept(x):
    """A tensor as a float64 array."""
    return x.detach().float().cpu().numpy().astype(np.float64)


def clipped(scales):
    """The scales as attention takes them."""
    s = scales.detach().double().cpu()
    return torch.where(s >= 2.0 ** -64, s, torch.full_like(s, 2.0 ** -64)).clamp(max=2.0 ** 64)


def dequantised(cache, scales):
    """A cache's values as float32 on the CPU (an attention reference takes them with a scale of 1)."""
    P, Hkv = scales.shape
    x = cache.detach().float().cpu().double().view(P, BS, Hkv, -1) * clipped(scales)[:, None, :, None]
    return x.view(P * BS, Hkv, -1).float()


def attention(q, kc, vc, ks, vs, table, rows, cu, seq_lens, prefix, sm_scale, topk=None, bq=1, cub=None):
    """(out, tolerance) of the prefill attention calls."""
    k, v = dequantised(kc, ks), dequantised(vc, vs)
    out, A = R.attention(q, k, v, table, rows, cu, seq_lens, prefix, sm_scale, 1.0, 1.0, topk, bq, cub)
    extra = _weights(q, k, vc, vs, table, rows, cu, seq_lens, prefix, sm_scale, topk, bq, cub)
    return out, A, 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -25 * 448 * extra[..., None]


def _weights(q, k, vc, vs, table, rows, cu, seq_lens, prefix, sm_scale, topk, bq, cub):
    """Keys read times the largest softmax weight x value scale, of each query row."""
    q, kc, vs = R.f64(q), R.f64(k), clipped(vs).numpy()
    table, rows, cu, seq_lens, prefix = (R.ints(x) for x in (table, rows, cu, seq_lens, prefix))
    T, Hq, _ = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    if topk is not None:
        topk, cub = R.ints(topk), R.ints(cub)
    out = np.zeros((T, Hq))
    for b in range(len(rows)):
        for t in range(cu[b], cu[b + 1]):
            i = t - cu[b]
            for h in range(Hkv):
                chosen = None
                if topk is not None:
                    r = cub[b] + i // bq
                    chosen = set(topk[h, r].tolist()) if r < min(cub[b + 1], topk.shape[1]) else set()
                s = R.readable(table, rows[b], kc.shape[0] // BS, min(prefix[b] + i + 1, seq_lens[b]), chosen)
                if len(s):
                    z = (q[t, h * G:(h + 1) * G] @ kc[s, h].T) * sm_scale
                    p = np.exp(z - z.max(-1, keepdims=True))
                    out[t, h * G:(h + 1) * G] = len(s) * (p / p.sum(-1, keepdims=True) * vs[s // BS, h]).max(-1)
    return out


def decode(q, kc, vc, ks, vs, table, seq_lens, req, sm_scale, topk=None):
    """(out, A, tolerance) of the decode calls: every row a chunk of one token."""
    T = q.shape[0]
    cu, lens = torch.arange(T + 1), seq_lens.cpu().long()
    lens = lens.clamp(min=0)
    return attention(q, kc, vc, ks, vs, table, req, cu, lens, (lens - 1).clamp(min=-1), sm_scale, topk, 1, cu if topk is not None else None)


def check_attention(got, ref, A, tol, what):
    got = R.f64(got)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), "%s: %d cells not finite" % (what, (~np.isfinite(got)).sum())
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), "%s: %d cells off, worst %.3g over its bound of %.3g (token %d)" % (
        what, (over > 0).sum(), over.max(), tol.flat[over.argmax()], np.unravel_index(over.argmax(), over.shape)[0])
    assert not got[A == 0].any(), what + ": a row that reads nothing is not zero"
