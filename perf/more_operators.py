"""The block-scaled 8-bit K/V cache of a serving loop, as measured work: its store and the attention that reads it.

The caches hold E4M3 codes with one fp32 scale for each page of 128 tokens and K/V head (`scales[page, head]`):

  store    paged_norm_rope_store_block_scaled: per-head RMS norm and rotary positions of queries and keys; K and V
           appended to their pages, whose scales grow with what comes in
  decode   paged_decode_attention_block_scaled / paged_sparse_decode_attention_block_scaled: single tokens and short
           runs of draft tokens over every page, or over the pages selected for each token
  prefill  paged_prefill_attention_block_scaled / paged_sparse_prefill_attention_block_scaled: ragged chunks

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` set calls the framework.  Heads,
pages, batches and lengths follow the package's workloads: 64 query heads over 8 K/V heads of 128 dims, up to 16384
tokens a request, 512-token chunks, and decode rows of 1, 4, 8 and 16 tokens.
"""
import math
import random

import torch

own = False

PAGE = 128
LIMIT = 17.2e9  # bytes of the plain form's 32-bit logits in the largest listed case
E4M3_MAX = 448.0
LEAST, MOST = -64, 64  # exponents of the scales that the store writes
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token of each of 16 requests: the store of a plain decode step, where latency counts
        {"name": "store_single", "op": "store", "seqs": 16, "rows": "one", "tokens": 16, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 128, "pairs": "halves", "type": "bf16", "context": 16384, "pad": 0, "lengths": 5},
        # draft tokens: 64 requests with 1, 4, 8 or 16 rows each, and the padding rows of a captured batch
        {"name": "store_drafts", "op": "store", "seqs": 64, "rows": "drafts", "tokens": 0, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 128, "pairs": "halves", "type": "bf16", "context": 16384, "pad": 24, "lengths": 6},
        # sixteen 512-token chunks at any offset: the store of a large prefill step
        {"name": "store_chunks", "op": "store", "seqs": 16, "rows": "even", "tokens": 8192, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 128, "pairs": "halves", "type": "bf16", "context": 16384, "pad": 0, "lengths": 4},
        # an odd number of tokens in chunks of any length, f16, half of each head rotated in neighbouring pairs
        {"name": "store_ragged_f16", "op": "store", "seqs": 7, "rows": "ragged", "tokens": 1999, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 64, "pairs": "neighbours", "type": "f16", "context": 9000, "pad": 5, "lengths": 7},
        # one token of one request of some 2000 tokens: the smallest call
        {"name": "decode_single", "op": "decode", "seqs": 1, "rows": "one", "tokens": 1, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 2048, "spread": "full", "topk": 0, "block_q": 1, "pad": 0, "lengths": 1},
        # the dense decode step: one token of each of 16 requests of 16384 tokens
        {"name": "decode_dense", "op": "decode", "seqs": 16, "rows": "one", "tokens": 16, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "full", "topk": 0, "block_q": 1, "pad": 0, "lengths": 2},
        # the verification step: 4 requests with 4 rows each over the 16 pages selected for each row
        {"name": "decode_verify", "op": "decode", "seqs": 4, "rows": "four", "tokens": 16, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "flat", "topk": 16, "block_q": 1, "pad": 0, "lengths": 3},
        # the mixed step: 64 requests with 1, 4, 8 or 16 rows over 64 selected pages, padding rows behind them
        {"name": "decode_mixed", "op": "decode", "seqs": 64, "rows": "drafts", "tokens": 0, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "log", "topk": 64, "block_q": 1, "pad": 9, "lengths": 6},
        # short chunks (16 tokens) of four long requests: few rows over a long cache
        {"name": "prefill_short", "op": "prefill", "seqs": 4, "rows": "even", "tokens": 64, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "flat", "topk": 0, "block_q": 0, "pad": 0, "lengths": 2},
        # ragged chunks of odd lengths with f16 queries, every key
        {"name": "prefill_ragged_f16", "op": "prefill", "seqs": 5, "rows": "ragged", "tokens": 1999, "hq": 64, "hkv": 8,
         "dim": 128, "type": "f16", "context": 9000, "spread": "log", "topk": 0, "block_q": 0, "pad": 0, "lengths": 8},
        # eight 512-token chunks at any offset, every key: the largest call
        {"name": "prefill_dense", "op": "prefill", "seqs": 8, "rows": "even", "tokens": 4096, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "flat", "topk": 0, "block_q": 0, "pad": 0, "lengths": 4},
        # the same chunks, each block of 64 tokens over the 32 pages selected for it
        {"name": "prefill_sparse", "op": "prefill", "seqs": 8, "rows": "even", "tokens": 4096, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "context": 16384, "spread": "flat", "topk": 32, "block_q": 64, "pad": 0, "lengths": 4},
    ]


def _log(rng, least, most):
    return max(least, min(most, round(math.exp(rng.uniform(math.log(least), math.log(most + 1))))))


def draw(rng):
    op = rng.choice(("store", "decode", "prefill"))
    hkv = rng.choice((1, 2, 4, 8))
    case = {"op": op, "hkv": hkv, "hq": hkv * rng.choice((1, 2, 4, 8, 8)), "dim": 128, "type": rng.choice(("bf16", "bf16", "bf16", "f16"))}
    if op == "store":
        case["dim"] = rng.choice((64, 128, 128))
        case["rot"], case["pairs"] = rng.choice((case["dim"], case["dim"] // 2)), rng.choice(("halves", "halves", "neighbours"))
        case["rows"] = rng.choice(("one", "drafts", "even", "ragged"))
        case["seqs"] = _log(rng, 1, 64)
        case["tokens"] = case["seqs"] if case["rows"] == "one" else _log(rng, case["seqs"], 8192)
        case["context"], case["pad"], case["lengths"] = _log(rng, 512, 16384), rng.choice((0, 0, 1, 17)), rng.randrange(1 << 20)
        return case
    while True:
        case["spread"], case["context"] = rng.choice(("flat", "log", "full")), _log(rng, 256, 16384)
        case["lengths"], case["pad"] = rng.randrange(1 << 20), rng.choice((0, 0, 3))
        case["topk"] = rng.choice((0, 4, 16, 33, 64))
        if op == "decode":
            case["rows"], case["seqs"], case["block_q"] = rng.choice(("one", "four", "drafts")), _log(rng, 1, 64), 1
            case["tokens"] = case["seqs"] * {"one": 1, "four": 4, "drafts": 0}[case["rows"]]
        else:
            case["dim"] = rng.choice((64, 128, 128))
            case["rows"], case["seqs"] = rng.choice(("even", "ragged")), _log(rng, 1, 12)
            case["tokens"] = _log(rng, case["seqs"], 4096)
            case["block_q"] = rng.choice((1, 16, 64, 100, 128)) if case["topk"] else 0
        if case["tokens"] > case["seqs"] * case["context"]:
            continue
        new, prefix = _lengths(case)
        if 4.0 * len(new) * max(new) * case["hq"] * max(n + p for n, p in zip(new, prefix)) <= LIMIT:
            return case


def _lengths(case):
    """New tokens and cached tokens of each request, from the case alone."""
    r = random.Random(case["lengths"])
    n, total, context = case["seqs"], case["tokens"], case["context"]
    if case["rows"] == "drafts":
        new = [r.choice((1, 4, 8, 16)) for _ in range(n)]
    elif case["rows"] == "ragged":
        share = [r.expovariate(1.0) for _ in range(n)]
        new = [1 + int((total - n) * s / sum(share)) for s in share]
        new[r.randrange(n)] += total - sum(new)
    else:
        new = [total // n + (i < total % n) for i in range(n)]
    new = [min(c, context) for c in new]
    spread = case.get("spread", "flat")
    if spread == "full":
        prefix = [context - c for c in new]
    elif spread == "flat":
        prefix = [r.randint(0, context - c) for c in new]
    else:
        whole = [int(math.exp(r.uniform(math.log(min(256, context)), math.log(context)))) for _ in new]
        prefix = [max(0, w - c) for w, c in zip(whole, new)]
    return new, prefix


def _blocks(n):
    return -(-n // PAGE)


# ----------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, seqs, owned, nb, spare_rows=2):
    """A page table with shuffled rows and scattered pages: (table, row of each request, pages of the pool).  Entries
    behind a request's last block name pages that it does not own."""
    need = sum(owned)
    pool = need + max(8, need // 8)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    rows = torch.randperm(seqs + spare_rows, generator=g, device="cuda")[:seqs]
    own_n = torch.tensor(owned, device="cuda")
    at = torch.cumsum(own_n, 0) - own_n
    j = torch.arange(nb, device="cuda")
    table = perm[torch.randint(0, pool, (seqs + spare_rows, nb), generator=g, device="cuda")]
    table[rows] = torch.where(j < own_n[:, None], perm[(at[:, None] + j).clamp(max=pool - 1)], table[rows])
    return table.contiguous(), rows.to(torch.int32), pool


def _scale_of(largest):
    """The smallest power of two that brings `largest` to at most 448, within the exponents that the store writes."""
    m, e = torch.frexp(largest.double() / E4M3_MAX)  # m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(largest > 0, e, LEAST).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(m), e).float()


def _cache(g, pool, heads, dim):
    """A cache whose pages and heads differ in magnitude, as those of a model's layers do, with its scales."""
    x = torch.randn((pool, PAGE, heads, dim), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((pool, 1, heads, 1), generator=g, device="cuda"))
    scales = _scale_of(x.abs().amax((1, 3)))
    x /= scales[:, None, :, None]
    return x.to(torch.float8_e4m3fn).view(pool * PAGE, heads, dim), scales


def prepare(case, seed):
    return _prepare_store(case, seed) if case["op"] == "store" else _prepare_attention(case, seed)


def _prepare_store(case, seed):
    g = _generator(seed)
    new, prefix = _lengths(case)
    hq, hkv, dim, rotary, kind = case["hq"], case["hkv"], case["dim"], case["rot"], TYPES[case["type"]]
    nb = _blocks(case["context"])
    whole = [n + p for n, p in zip(new, prefix)]
    table, rows, pool = _table(g, len(new), [_blocks(n) for n in whole], nb)
    # queries, keys and values are slices of one projection's output, whose heads differ in magnitude
    t = sum(new) + case["pad"]
    fused = torch.randn((t, hq + 2 * hkv, dim), generator=g, device="cuda")
    fused *= torch.exp(0.7 * torch.randn((1, hq + 2 * hkv, 1), generator=g, device="cuda"))
    fused = fused.to(kind)
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
    cu = torch.tensor([0] + new, device="cuda").cumsum(0)
    pos = torch.tensor(prefix, device="cuda")[seq] + torch.arange(sum(new), device="cuda") - cu[seq]
    slots = table[rows.long()[seq], pos // PAGE].long() * PAGE + pos % PAGE
    fill = torch.zeros(case["pad"], device="cuda", dtype=torch.int64)
    # the parts of each request's pages that its tokens fill, as its scheduler knows them: first row, rows, offset
    parts, row = [], 0
    for n, p in zip(new, prefix):
        while n > 0:
            take = min(n, PAGE - p % PAGE)
            parts.append((row, take, p % PAGE))
            row, n, p = row + take, n - take, p + take
    half = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(case["context"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * half / rotary)
    k_cache, k_scales = _cache(g, pool, hkv, dim)
    v_cache, v_scales = _cache(g, pool, hkv, dim)
    return {"case": case, "q": fused[:, :hq], "k": fused[:, hq:hq + hkv], "v": fused[:, hq + hkv:],
            "wq": (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(kind),
            "wk": (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(kind),
            "cos_sin": torch.cat((angle.cos(), angle.sin()), 1).float(), "eps": 1e-6,
            "lens": torch.cat((pos + 1, fill)).to(torch.int32), "slots": torch.cat((slots, fill - 1)).to(torch.int32),
            "first": torch.tensor([x[0] for x in parts], device="cuda"), "count": torch.tensor([x[1] for x in parts], device="cuda"),
            "offset": torch.tensor([x[2] for x in parts], device="cuda"),
            "out": torch.empty((t, hq, dim), dtype=kind, device="cuda"),
            "k_cache": k_cache, "k_scales": k_scales, "v_cache": v_cache, "v_scales": v_scales}


def _prepare_attention(case, seed):
    g = _generator(seed)
    new, prefix = _lengths(case)
    seqs, hq, hkv, dim = case["seqs"], case["hq"], case["hkv"], case["dim"]
    nb = _blocks(case["context"])
    whole = [n + p for n, p in zip(new, prefix)]
    table, rows, pool = _table(g, seqs, [_blocks(n) for n in whole], nb)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    t = cu[-1] + case["pad"]  # rows behind the last request are padding
    seq = [b for b, n in enumerate(new) for _ in range(n)]
    state = {"case": case, "table": table, "rows": rows, "cu": _int32(cu), "seq_lens": _int32(whole), "prefix": _int32(prefix),
             "req": torch.cat((rows[torch.tensor(seq, device="cuda")], _int32([-1] * case["pad"]))),
             "lens": _int32([p + i + 1 for n, p in zip(new, prefix) for i in range(n)] + [0] * case["pad"]),
             "q": torch.randn((t, hq, dim), generator=g, device="cuda").to(TYPES[case["type"]]),
             "out": torch.empty((t, hq, dim), dtype=torch.bfloat16, device="cuda"), "sm_scale": dim ** -0.5,
             "longest": max(new), "most": max(whole)}
    state["k_cache"], state["k_scales"] = _cache(g, pool, hkv, dim)
    state["v_cache"], state["v_scales"] = _cache(g, pool, hkv, dim)
    if case["topk"]:
        # what the selection in front gives: the first and the last two visible blocks, then the best of the others
        bq, top = case["block_q"], case["topk"]
        cub = [0]
        for n in new:
            cub.append(cub[-1] + -(-n // bq))
        seen = [_blocks(min(p + q * bq + 1, w)) for n, p, w in zip(new, prefix, whole) for q in range(-(-n // bq))]
        seen = torch.tensor(seen, device="cuda")[:, None]
        j = torch.arange(nb, device="cuda")
        score = torch.rand((cub[-1], nb), generator=g, device="cuda")
        score = torch.where((j < 1) | (j >= seen - 2), 2.0 + score, score)
        best, ids = torch.where(j < seen, score, -1.0).topk(min(top, nb), dim=1)
        pick = torch.full((1, cub[-1] + (case["pad"] if case["op"] == "decode" else 0), top), -1, dtype=torch.int32, device="cuda")
        pick[0, :cub[-1], :ids.shape[1]] = torch.where(best >= 0, ids, -1).to(torch.int32)
        state["topk"], state["cu_blocks"] = pick.expand(hkv, -1, -1), _int32(cub)
    return state


# -------------------------------------------------------------------- run


def run(state):
    return _store(state) if state["case"]["op"] == "store" else _attention(state)


def _turned(x, cos, sin, pairs):
    """The rotated dims [T, heads, rot] of x by each token's angles [T, 1, rot / 2]."""
    if pairs == "halves":
        a, b = x.chunk(2, dim=-1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)


def _normed_turned(x, w, s):
    rotary = s["case"]["rot"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    row = s["cos_sin"][(s["lens"].long() - 1).clamp(min=0)][:, None]
    cos, sin = row.chunk(2, dim=-1)
    return torch.cat((_turned(x[..., :rotary], cos, sin, s["case"]["pairs"]), x[..., rotary:]), -1)


def _append(cache, scales, values, s):
    """Values [T, heads, dim] into the pages that their slots name, each page's scales grown to hold them."""
    live = values.shape[0] - s["case"]["pad"]
    values, slots = values[:live], s["slots"][:live].long()
    part = torch.repeat_interleave(torch.arange(s["first"].numel(), device=slots.device), s["count"], output_size=live)
    page = slots[s["first"]] // PAGE
    largest = torch.zeros((s["first"].numel(), values.shape[1]), device=slots.device)
    largest.scatter_reduce_(0, part[:, None].expand(-1, values.shape[1]), values.abs().amax(-1), "amax")
    need = _scale_of(largest)
    old = torch.where(s["offset"][:, None] > 0, scales[page], 0.0)  # a page's first token starts its scales anew
    scale = torch.maximum(old, need)
    # the tokens that a page holds already, at the scale that it has now
    pages = cache.view(-1, PAGE, *cache.shape[1:])
    held = torch.arange(PAGE, device=slots.device) < s["offset"][:, None]
    before = pages[page].float()
    ratio = torch.where(held[:, :, None], (old / scale)[:, None], 1.0)
    pages.view(torch.uint8)[page] = (before * ratio[..., None]).to(cache.dtype).view(torch.uint8)
    scales[page] = scale
    codes = (values / scale[part][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
    cache.view(torch.uint8)[slots] = codes.view(torch.uint8)


def _store(s):
    if own:
        import sparse_paged_decode_gb300 as spd

        spd.paged_norm_rope_store_block_scaled(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos_sin"], s["lens"], s["slots"],
                                               s["out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["eps"],
                                               s["case"]["pairs"] == "neighbours", PAGE)
        return s["out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    q = _normed_turned(s["q"], s["wq"], s)
    _append(s["k_cache"], s["k_scales"], _normed_turned(s["k"], s["wk"], s), s)
    _append(s["v_cache"], s["v_scales"], s["v"].float(), s)
    q = torch.where(s["lens"][:, None, None] > 0, q, 0.0)
    return q.to(s["q"].dtype), s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _attention(s):
    case = s["case"]
    if own:
        import sparse_paged_decode_gb300 as spd

        t, nb = s["q"].shape[0], s["table"].shape[1]
        if "workspace" not in s:  # a program keeps its workspace between calls
            if case["op"] == "decode":
                size = spd.decode_workspace_bytes(t, case["hq"], case["hkv"], case["dim"], nb)
            else:
                size = spd.prefill_attention_workspace_bytes(t, case["hq"], case["hkv"], case["dim"], case["seqs"], nb,
                                                             s["topk"].shape[1] if case["topk"] else 0)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        cache = (s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"])
        last = (s["out"], s["sm_scale"], PAGE, s["workspace"])
        if case["op"] == "decode":
            if case["topk"]:
                spd.paged_sparse_decode_attention_block_scaled(*cache, s["lens"], s["req"], s["topk"], *last)
            else:
                spd.paged_decode_attention_block_scaled(*cache, s["lens"], s["req"], *last)
        elif case["topk"]:
            spd.paged_sparse_prefill_attention_block_scaled(*cache, s["rows"], s["cu"], s["seq_lens"], s["prefix"], s["topk"],
                                                            case["block_q"], s["cu_blocks"], *last)
        else:
            spd.paged_prefill_attention_block_scaled(*cache, s["rows"], s["cu"], s["seq_lens"], s["prefix"], *last)
        return s["out"]
    q, cu, prefix, seq_lens = s["q"], s["cu"].long(), s["prefix"].long(), s["seq_lens"].long()
    t, hq, dim = q.shape
    seqs, hkv, g = prefix.numel(), case["hkv"], hq // case["hkv"]
    nb = _blocks(s["most"])
    width, keys = s["longest"], nb * PAGE
    # requests side by side, padded to the longest chunk and the longest request
    i = torch.arange(width, device=q.device)
    token = (cu[:-1, None] + i).clamp(max=t - 1)
    qs = q[token].float().view(seqs, width, hkv, g, dim).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, width * g, dim)
    pages = s["table"][s["rows"].long(), :nb].long()

    def gathered(cache, scales):
        x = cache.view(-1, PAGE, hkv, dim)[pages].float()
        return x.mul_(scales[pages][:, :, None, :, None]).view(seqs, keys, hkv, dim)

    ks = gathered(s["k_cache"], s["k_scales"]).permute(0, 2, 3, 1)
    z = (qs * s["sm_scale"]) @ ks
    del ks
    pos = prefix[:, None] + i
    key = torch.arange(keys, device=q.device)
    hidden = (key > pos[..., None]) | (key >= seq_lens[:, None, None])  # [seqs, width, keys]
    if case["topk"]:
        row = (s["cu_blocks"].long()[:-1, None] + i // case["block_q"]).clamp(max=s["topk"].shape[1] - 1)
        ids = s["topk"][0].long()
        # ids past the last listed block share a column of their own, which is dropped
        take = torch.zeros((ids.shape[0], nb + 1), dtype=torch.bool, device=q.device)
        take.scatter_(1, torch.where((ids >= 0) & (ids < nb), ids, nb), True)
        hidden = hidden | ~take[:, :nb][row].repeat_interleave(PAGE, dim=2)
    z = z.view(seqs, hkv, width, g, keys).masked_fill_(hidden[:, None, :, None], float("-inf"))
    top = z.amax(-1, keepdim=True)
    z.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = z.sum(-1, keepdim=True)
    vs = gathered(s["v_cache"], s["v_scales"]).permute(0, 2, 1, 3)
    o = (z.view(seqs, hkv, width * g, keys) @ vs).view(seqs, hkv, width, g, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(seqs, width, hq, dim)
    of = torch.arange(t, device=q.device)
    b = torch.searchsorted(cu[1:], of, right=True).clamp(max=seqs - 1)
    o = o[b, (of - cu[b]).clamp(max=width - 1)]
    return torch.where((of < cu[-1])[:, None, None], o, 0.0).to(torch.bfloat16)


# ------------------------------------------------------------------- work


def work(case):
    new, prefix = _lengths(case)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    tokens = sum(new)
    if case["op"] == "store":
        touched = sum(_blocks(n + p) - p // PAGE for n, p in zip(new, prefix))
        # q in and out, k and v in, their codes out, the angles; length and slot of each row; the pages' scales in and out
        values = 4 * hq * dim + 2 * hkv * dim * (2 + 1)
        return {"bytes": float(tokens * (values + 8 + 4 * case["rot"]) + 4 * dim + 16 * touched * hkv),
                "flops": float(tokens * ((hq + hkv) * (5 * dim + 3 * case["rot"]) + 2 * hkv * dim * 2))}
    pairs, read = 0, 0
    for n, p in zip(new, prefix):
        if not case["topk"]:
            pairs += n * p + n * (n + 1) // 2
            read += p + n
            continue
        bq, top = case["block_q"], case["topk"]
        for q in range(-(-n // bq)):
            seen = p + q * bq + 1
            span = min(bq, n - q * bq)
            last = seen - (_blocks(seen) - 1) * PAGE  # keys of the last selected block below the first token's position
            whole = min(top, _blocks(seen)) - 1
            pairs += sum(whole * PAGE + min(PAGE, last + i) for i in range(span))
        blocks = min(_blocks(p + n), top * -(-n // bq))  # at least these pages are read by a selection of this width
        read += min(p + n, max(min(top, blocks), 1) * PAGE)
    table = sum(_blocks(n + p) for n, p in zip(new, prefix))
    picked = 4 * case["topk"] * sum(-(-n // case["block_q"]) for n in new) if case["topk"] else 0
    return {"bytes": 4.0 * tokens * hq * dim + 2.0 * read * hkv * (dim + 4 / PAGE) + 4.0 * table + picked,
            "flops": 4.0 * pairs * hq * dim}


# ------------------------------------------------------------------ exact


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attention(s)


def _exact_store(s):
    """Each head as complex numbers, the rotation a product with e^(i position angle); page by page, each with its scale."""
    case = s["case"]
    rotary, pos = case["rot"], (s["lens"].double() - 1).clamp(min=0)
    wave = 10000.0 ** (-torch.arange(0, rotary, 2, device="cuda").double() / rotary)
    turn = torch.exp(1j * pos[:, None] * wave)

    def one(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
        half = rotary // 2
        lead = (torch.complex(x[..., :half].contiguous(), x[..., half:rotary].contiguous()) if case["pairs"] == "halves"
                else torch.view_as_complex(x[..., :rotary].reshape(*x.shape[:-1], half, 2).contiguous()))
        lead = lead * turn[:, None]
        if case["pairs"] == "halves":
            x[..., :half], x[..., half:rotary] = lead.real, lead.imag
        else:
            x[..., 0:rotary:2], x[..., 1:rotary:2] = lead.real, lead.imag
        return x

    def appended(cache, scales, x):
        cache, scales = cache.double(), scales.double()
        slots = s["slots"].tolist()
        for first, count, offset in zip(s["first"].tolist(), s["count"].tolist(), s["offset"].tolist()):
            page, fresh = slots[first] // PAGE, x[first:first + count]
            least = fresh.abs().amax((0, 2)) / E4M3_MAX
            grown = torch.exp2(torch.ceil(torch.log2(least)).clamp(LEAST, MOST))
            before = scales[page].clone() if offset else torch.zeros_like(grown)
            scales[page] = torch.where(before >= grown, before, grown)
            held = slice(page * PAGE, page * PAGE + offset)
            cache[held] *= (before / scales[page])[:, None]
            cache[slots[first]:slots[first] + count] = fresh / scales[page][:, None]
        return cache, scales

    q = one(s["q"], s["wq"])
    q[s["lens"] <= 0] = 0.0
    k, ks = appended(s["k_cache"], s["k_scales"], one(s["k"], s["wk"]))
    v, vs = appended(s["v_cache"], s["v_scales"], s["v"].double())
    return q, k, v, ks, vs


def _exact_attention(s):
    """Request by request and head by head, with each request's keys in their own order."""
    case = s["case"]
    cu, lens, prefix = s["cu"].tolist(), s["seq_lens"].tolist(), s["prefix"].tolist()
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (length, before) in enumerate(zip(lens, prefix)):
        at = torch.arange(length, device="cuda")
        page = s["table"][s["rows"][b].long()].long()[at // PAGE]
        slot = page * PAGE + at % PAGE
        n = cu[b + 1] - cu[b]
        seen = at[None, :] <= before + torch.arange(n, device="cuda")[:, None]
        if case["topk"]:
            lo = s["cu_blocks"].tolist()
            ids = s["topk"][0, lo[b]:lo[b + 1]]
            listed_ = torch.stack([(ids == j).any(1) for j in range(_blocks(length))], 1)
            seen = seen & listed_.repeat_interleave(case["block_q"], 0)[:n].repeat_interleave(PAGE, 1)[:, :length]
        for h in range(hkv):
            k = s["k_cache"][slot, h].double() * s["k_scales"][page, h, None].double()
            v = s["v_cache"][slot, h].double() * s["v_scales"][page, h, None].double()
            q = s["q"][cu[b]:cu[b + 1], h * g:(h + 1) * g].double()
            z = torch.einsum("tgd,kd->tgk", q, k) * s["sm_scale"]
            z = torch.where(seen[:, None], z, -torch.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)  # a row that sees no key is zero
            out[cu[b]:cu[b + 1], h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", p, v)
    return out
