"""The serving-step operators in front of and behind the paged K/V cache, as measured work.

Three operators of one serving step over the paged cache, in the order in which the step calls them:

  assign     paged_assign_slots: page-table rows grown from the free list, and every token's row, length and slot
  store      paged_norm_rope_store: per-head RMS norm and rotary positions of queries and keys, K and V into the cache
  attention  paged_prefill_attention / paged_sparse_prefill_attention: ragged chunks of new tokens over the cache

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` set calls the framework.  Heads,
pages and lengths follow the package's workloads: 64 query heads over 8 K/V heads of 128 dims, pages of 128 tokens,
up to 16384 tokens a request, 512-token chunks, and decode rows of 1, 4, 8 and 16 tokens.
"""
import math
import random

import torch

own = False

PAGE = 128
LIMIT = 17.2e9  # bytes of the plain form's 32-bit logits in the largest listed case
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step of 64 requests with 1, 4, 8 or 16 tokens each: the latency of a small call
        {"name": "assign_decode", "op": "assign", "seqs": 64, "tokens": 466, "context": 16384, "spread": "log",
         "even": False, "block_q": 1, "lengths": 5},
        # a prefill step: eight chunks of 512 tokens at any offset of a 16384-token request
        {"name": "assign_prefill", "op": "assign", "seqs": 8, "tokens": 4096, "context": 16384, "spread": "flat",
         "even": True, "block_q": 64, "lengths": 4},
        # a wide step: a thousand requests, chunks and single tokens mixed
        {"name": "assign_wide", "op": "assign", "seqs": 1024, "tokens": 65536, "context": 16384, "spread": "log",
         "even": False, "block_q": 64, "lengths": 6},
        # decode rows into the FP8 cache: few tokens, latency
        {"name": "store_decode_e4m3", "op": "store", "tokens": 466, "hq": 64, "hkv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "cache": "e4m3", "values": True, "context": 16384, "lengths": 5},
        # a large prefill step into the FP8 cache
        {"name": "store_prefill_e4m3", "op": "store", "tokens": 8192, "hq": 64, "hkv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "cache": "e4m3", "values": True, "context": 16384, "lengths": 4},
        # an odd number of tokens into the BF16 cache, half of each head rotated in neighbouring pairs
        {"name": "store_ragged_bf16", "op": "store", "tokens": 1999, "hq": 64, "hkv": 8, "dim": 128, "rot": 64,
         "pairs": "neighbours", "cache": "bf16", "values": True, "context": 16384, "lengths": 7},
        # index queries and the index key of a prefill step: one head each, no values
        {"name": "store_index_bf16", "op": "store", "tokens": 4096, "hq": 1, "hkv": 1, "dim": 128, "rot": 128,
         "pairs": "halves", "cache": "bf16", "values": False, "context": 16384, "lengths": 4},
        # short chunks (16 tokens) of four long requests: few rows over a long cache
        {"name": "attend_short_e4m3", "op": "attention", "seqs": 4, "tokens": 64, "hq": 64, "hkv": 8, "dim": 128,
         "cache": "e4m3", "context": 16384, "spread": "flat", "even": True, "block_q": 0, "topk": 0, "lengths": 2},
        # eight 512-token chunks at any offset over the BF16 cache, every key
        {"name": "attend_prefill_bf16", "op": "attention", "seqs": 8, "tokens": 4096, "hq": 64, "hkv": 8, "dim": 128,
         "cache": "bf16", "context": 16384, "spread": "flat", "even": True, "block_q": 0, "topk": 0, "lengths": 4},
        # ragged chunks of odd lengths over the FP8 cache, every key
        {"name": "attend_ragged_e4m3", "op": "attention", "seqs": 5, "tokens": 1999, "hq": 64, "hkv": 8, "dim": 128,
         "cache": "e4m3", "context": 9000, "spread": "log", "even": False, "block_q": 0, "topk": 0, "lengths": 8},
        # the eight chunks over the FP8 cache, each block of 64 tokens over the 32 key blocks selected for it
        {"name": "attend_sparse_e4m3", "op": "attention", "seqs": 8, "tokens": 4096, "hq": 64, "hkv": 8, "dim": 128,
         "cache": "e4m3", "context": 16384, "spread": "flat", "even": True, "block_q": 64, "topk": 32, "lengths": 4},
        # ragged chunks over the BF16 cache with small query blocks, so that neighbours' selections differ
        {"name": "attend_sparse_bf16", "op": "attention", "seqs": 6, "tokens": 1111, "hq": 64, "hkv": 8, "dim": 128,
         "cache": "bf16", "context": 16384, "spread": "log", "even": False, "block_q": 16, "topk": 16, "lengths": 9},
    ]


def _log(rng, least, most):
    return max(least, min(most, round(math.exp(rng.uniform(math.log(least), math.log(most + 1))))))


def draw(rng):
    op = rng.choice(("assign", "store", "attention"))
    lengths = rng.randrange(1 << 20)
    if op == "assign":
        seqs = _log(rng, 1, 1024)
        return {"op": op, "seqs": seqs, "tokens": _log(rng, seqs, 65536), "context": _log(rng, 256, 16384),
                "spread": rng.choice(("flat", "log")), "even": rng.random() < 0.3,
                "block_q": rng.choice((1, 3, 16, 64, 128)), "lengths": lengths}
    dim = rng.choice((64, 128, 128, 128))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 8, 8))
    cache = rng.choice(("e4m3", "bf16"))
    if op == "store":
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hq, "hkv": hkv, "dim": dim,
                "rot": rng.choice((dim, dim // 2)), "pairs": rng.choice(("halves", "halves", "neighbours")),
                "cache": cache, "values": rng.random() < 0.8, "context": _log(rng, 512, 16384), "lengths": lengths}
    while True:
        seqs = rng.randint(1, 12)
        sparse = rng.random() < 0.5
        case = {"op": op, "seqs": seqs, "tokens": _log(rng, seqs, 4096), "hq": hq, "hkv": hkv, "dim": dim,
                "cache": cache, "context": _log(rng, 256, 16384), "spread": rng.choice(("flat", "log")),
                "even": rng.random() < 0.3, "block_q": rng.choice((1, 16, 64, 100, 128)) if sparse else 0,
                "topk": rng.choice((4, 16, 32, 33)) if sparse else 0, "lengths": rng.randrange(1 << 20)}
        if case["tokens"] > seqs * case["context"]:
            continue
        new, prefix = _lengths(case)
        if 4.0 * seqs * max(new) * hq * max(n + p for n, p in zip(new, prefix)) <= LIMIT:
            return case


def _lengths(case):
    """New tokens and cached tokens of each request, from the case alone."""
    r = random.Random(case["lengths"])
    n, total, context = case["seqs"], case["tokens"], case["context"]
    if case["even"]:
        new = [total // n + (i < total % n) for i in range(n)]
    else:
        share = [r.expovariate(1.0) for _ in range(n)]
        new = [1 + int((total - n) * s / sum(share)) for s in share]
        new[r.randrange(n)] += total - sum(new)
    new = [min(c, context) for c in new]
    if case["spread"] == "flat":
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
    """A page table with shuffled rows and scattered pages: (table, row of each request, pages of the pool, free pages).
    Entries behind a request's last block name pages that it does not own."""
    need = sum(owned)
    pool = need + max(8, need // 8)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    rows = torch.randperm(seqs + spare_rows, generator=g, device="cuda")[:seqs]
    own_n = torch.tensor(owned, device="cuda")
    at = torch.cumsum(own_n, 0) - own_n
    j = torch.arange(nb, device="cuda")
    mine = j < own_n[:, None]
    other = torch.randint(0, pool, (seqs + spare_rows, nb), generator=g, device="cuda")
    table = perm[other]
    table[rows] = torch.where(mine, perm[(at[:, None] + j).clamp(max=pool - 1)], table[rows])
    return table.contiguous(), rows.to(torch.int32), pool, perm[need:].contiguous()


def _cache(g, pool, heads, dim, kind):
    """A K or V cache with values in every slot and its static scale."""
    x = torch.randn((pool * PAGE, heads, dim), generator=g, device="cuda")
    if kind == "bf16":
        return x.to(torch.bfloat16), 1.0
    scale = float(x.abs().max()) / E4M3_MAX
    return (x / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    return {"assign": _prepare_assign, "store": _prepare_store, "attention": _prepare_attention}[case["op"]](case, seed)


def _prepare_assign(case, seed):
    g = _generator(seed)
    new, prefix = _lengths(case)
    nb = _blocks(case["context"])
    cached = [_blocks(p) for p in prefix]
    grown = sum(_blocks(p + n) for n, p in zip(new, prefix)) - sum(cached)
    table, rows, pool, _ = _table(g, case["seqs"], cached, nb)
    pool += grown + 16
    free = torch.randperm(grown + 16, generator=g, device="cuda").to(torch.int32) + (pool - grown - 16)
    seqs, tokens = case["seqs"], case["tokens"] + 8  # the last 8 token rows are padding
    return {"case": case, "new": _int32(new), "prefix": _int32(prefix), "rows": rows, "table": table, "free": free,
            "count": _int32([grown + 16]), "pool": pool, "cu": _int32([0] * (seqs + 1)),
            "cu_blocks": _int32([0] * (seqs + 1)), "seq_lens": _int32([0] * seqs), "req": _int32([0] * tokens),
            "lens": _int32([0] * tokens), "slots": _int32([0] * tokens), "left": _int32([0])}


def _prepare_store(case, seed):
    g = _generator(seed)
    t, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
    rotary, parts = case["rot"], hq + (2 if case["values"] else 1) * hkv
    # queries, keys and values are slices of one projection's output
    fused = torch.randn((t, parts, dim), generator=g, device="cuda").to(torch.bfloat16)
    pool = max(64, 2 * _blocks(t))
    # requests' tokens fill pages in order; one token in twenty is padding of a captured batch
    perm = torch.randperm(pool, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    slots = perm[i // PAGE] * PAGE + i % PAGE
    chunk = random.Random(case["lengths"]).randint(1, 512)
    offset = torch.randint(0, max(1, case["context"] - chunk + 1), (-(-t // chunk),), generator=g, device="cuda")
    lens = (offset[i // chunk] + i % chunk + 1).clamp(max=case["context"])
    pad = torch.rand(t, generator=g, device="cuda") < 0.05
    pad[0] = False
    half = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(case["context"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * half / rotary)
    k_cache, k_scale = _cache(g, pool, hkv, dim, case["cache"])
    state = {"case": case, "q": fused[:, :hq], "k": fused[:, hq:hq + hkv], "v": None, "v_cache": None, "v_scale": 1.0,
             "wq": (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16),
             "wk": (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16),
             "cos_sin": torch.cat((angle.cos(), angle.sin()), 1).float(), "eps": 1e-6,
             "lens": torch.where(pad, 0, lens).to(torch.int32), "slots": torch.where(pad, -1, slots).to(torch.int32),
             "out": torch.empty((t, hq, dim), dtype=torch.bfloat16, device="cuda"), "k_cache": k_cache, "k_scale": k_scale}
    if case["values"]:
        state["v"] = fused[:, hq + hkv:]
        state["v_cache"], state["v_scale"] = _cache(g, pool, hkv, dim, case["cache"])
    return state


def _prepare_attention(case, seed):
    g = _generator(seed)
    new, prefix = _lengths(case)
    seqs, hq, hkv, dim = case["seqs"], case["hq"], case["hkv"], case["dim"]
    nb = _blocks(case["context"])
    whole = [n + p for n, p in zip(new, prefix)]
    table, rows, pool, _ = _table(g, seqs, [_blocks(n) for n in whole], nb)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state = {"case": case, "table": table, "rows": rows, "cu": _int32(cu), "seq_lens": _int32(whole), "prefix": _int32(prefix),
             "q": torch.randn((cu[-1], hq, dim), generator=g, device="cuda").to(torch.bfloat16),
             "out": torch.empty((cu[-1], hq, dim), dtype=torch.bfloat16, device="cuda"), "sm_scale": dim ** -0.5,
             "longest": max(new), "most": max(whole)}
    state["k_cache"], state["k_scale"] = _cache(g, pool, hkv, dim, case["cache"])
    state["v_cache"], state["v_scale"] = _cache(g, pool, hkv, dim, case["cache"])
    if case["block_q"]:
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
        ids = torch.where(best >= 0, ids, -1).to(torch.int32)
        pick = torch.full((1, cub[-1], top), -1, dtype=torch.int32, device="cuda")
        pick[0, :, :ids.shape[1]] = ids
        state["topk"], state["cu_blocks"] = pick.expand(hkv, -1, -1), _int32(cub)
    return state


# -------------------------------------------------------------------- run


def run(state):
    return {"assign": _assign, "store": _store, "attention": _attention}[state["case"]["op"]](state)


def _assign(s):
    if own:
        import sparse_paged_decode_gb300 as spd

        spd.paged_assign_slots(s["new"], s["prefix"], s["rows"], s["free"], s["count"], s["pool"], PAGE,
                               s["case"]["block_q"], s["table"], s["cu"], s["cu_blocks"], s["seq_lens"], s["req"],
                               s["lens"], s["slots"], s["left"])
        return tuple(s[k] for k in ("table", "cu", "cu_blocks", "seq_lens", "req", "lens", "slots", "left"))
    new, prefix, rows, table = s["new"].long(), s["prefix"].long(), s["rows"].long(), s["table"]
    nb, dev = table.shape[1], table.device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    cu = torch.cat((zero, new.cumsum(0)))
    bq = s["case"]["block_q"]
    cu_blocks = torch.cat((zero, ((new + bq - 1) // bq).cumsum(0)))
    whole = prefix + new
    first = (prefix + PAGE - 1) // PAGE
    need = (whole + PAGE - 1) // PAGE - first
    at = torch.cat((zero, need.cumsum(0)))
    # grown blocks, as many as there can be: the last free page goes first
    i = torch.arange(s["req"].numel() // PAGE + new.numel() + 1, device=dev)
    b = torch.searchsorted(at[1:], i, right=True).clamp(max=new.numel() - 1)
    count = s["count"].long()
    page = torch.where(i < count, s["free"][(count - 1 - i).clamp(0, s["free"].numel() - 1)], -1).to(torch.int32)
    cell = torch.where(i < at[-1], rows[b] * nb + first[b] + i - at[b], table.numel())
    grown = torch.cat((table.view(-1), table.new_zeros(1)))
    grown[cell] = page
    table.copy_(grown[:-1].view_as(table))
    # every token's row, length and slot
    t = torch.arange(s["req"].numel(), device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=new.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, prefix[b] + t - cu[b], 0)
    page = table[rows[b], pos // PAGE].long()
    slot = torch.where(live & (page >= 0), page * PAGE + pos % PAGE, -1)
    i32 = torch.int32
    return (table, cu.to(i32), cu_blocks.to(i32), whole.to(i32), torch.where(live, rows[b], -1).to(i32),
            torch.where(live, pos + 1, 0).to(i32), slot.to(i32), (count - at[-1]).clamp(min=0).to(i32))


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


def _put(cache, values, scale, s):
    live = s["slots"] >= 0
    token = torch.arange(live.numel(), device=live.device)
    token = torch.where(live, token, live.int().argmax())  # padding writes a stored token's values once more
    if cache.dtype == torch.float8_e4m3fn:
        codes = (values / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        cache.view(torch.uint8)[s["slots"].long()[token]] = codes.view(torch.uint8)[token]
    else:
        cache[s["slots"].long()[token]] = values.to(cache.dtype)[token]


def _store(s):
    if own:
        import sparse_paged_decode_gb300 as spd

        spd.paged_norm_rope_store(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos_sin"], s["lens"], s["slots"], s["out"],
                                  s["k_cache"], s["v_cache"], s["eps"], s["case"]["pairs"] == "neighbours", PAGE,
                                  s["k_scale"], s["v_scale"])
        return s["out"], s["k_cache"], s["v_cache"]
    q = _normed_turned(s["q"], s["wq"], s)
    _put(s["k_cache"], _normed_turned(s["k"], s["wk"], s), s["k_scale"], s)
    if s["v"] is not None:
        _put(s["v_cache"], s["v"].float(), s["v_scale"], s)
    q = torch.where(s["lens"][:, None, None] > 0, q, 0.0)
    return q.to(torch.bfloat16), s["k_cache"], s["v_cache"]


def _attention(s):
    case = s["case"]
    if own:
        import sparse_paged_decode_gb300 as spd

        if "workspace" not in s:  # a program keeps its workspace between calls
            rows = s["topk"].shape[1] if case["block_q"] else 0
            size = spd.prefill_attention_workspace_bytes(s["q"].shape[0], case["hq"], case["hkv"], case["dim"], case["seqs"],
                                                         s["table"].shape[1], rows)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        common = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["rows"], s["cu"], s["seq_lens"], s["prefix"])
        scales = (s["sm_scale"], PAGE, s["k_scale"], s["v_scale"], s["workspace"])
        if case["block_q"]:
            spd.paged_sparse_prefill_attention(*common, s["topk"], case["block_q"], s["cu_blocks"], s["out"], *scales)
        else:
            spd.paged_prefill_attention(*common, s["out"], *scales)
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
    ks = s["k_cache"].view(-1, PAGE, hkv, dim)[pages].float().view(seqs, keys, hkv, dim).permute(0, 2, 3, 1)
    z = (qs * (s["sm_scale"] * s["k_scale"])) @ ks
    del ks
    pos = prefix[:, None] + i
    key = torch.arange(keys, device=q.device)
    hidden = (key > pos[..., None]) | (key >= seq_lens[:, None, None])  # [seqs, width, keys]
    if case["block_q"]:
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
    vs = s["v_cache"].view(-1, PAGE, hkv, dim)[pages].float().view(seqs, keys, hkv, dim).permute(0, 2, 1, 3)
    o = (z.view(seqs, hkv, width * g, keys) @ vs).view(seqs, hkv, width, g, dim)
    o = torch.where(total > 0, o * s["v_scale"] / total, 0.0).permute(0, 2, 1, 3, 4).reshape(seqs, width, hq, dim)
    of = torch.arange(t, device=q.device)
    b = torch.searchsorted(cu[1:], of, right=True)
    return o[b, of - cu[b]].to(torch.bfloat16)


# ------------------------------------------------------------------- work


def work(case):
    if case["op"] == "assign":
        new, prefix = _lengths(case)
        first = sum(_blocks(p) for p in prefix)
        grown = sum(_blocks(p + n) for n, p in zip(new, prefix)) - first
        # lengths and rows in; the grown pages in and out; offsets, lengths and the tokens' three numbers out; the
        # page of each partly filled block
        return {"bytes": 4.0 * (6 * case["seqs"] + 2 * grown + 3 * (case["tokens"] + 8) + 4 + case["seqs"]), "flops": 0.0}
    if case["op"] == "store":
        t, hq, hkv, dim, rotary = (case[k] for k in ("tokens", "hq", "hkv", "dim", "rot"))
        size = 1 if case["cache"] == "e4m3" else 2
        kv = 2 if case["values"] else 1
        values = 4 * hq * dim + kv * hkv * dim * (2 + size)
        return {"bytes": float(t * (values + 8 + 4 * rotary) + 4 * dim), "flops": float(t * (hq + hkv) * (5 * dim + 3 * rotary))}
    new, prefix = _lengths(case)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    size = 1 if case["cache"] == "e4m3" else 2
    pairs, read = 0, 0
    for n, p in zip(new, prefix):
        if not case["block_q"]:
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
    tokens = sum(new)
    table = sum(_blocks(n + p) for n, p in zip(new, prefix))
    picked = 4 * case["topk"] * sum(-(-n // case["block_q"]) for n in new) if case["block_q"] else 0
    return {"bytes": 4.0 * tokens * hq * dim + 2.0 * read * hkv * dim * size + 4.0 * table + picked,
            "flops": 4.0 * pairs * hq * dim}


# ------------------------------------------------------------------ exact


def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers: the plain form's are the definition's
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attention(s)


def _exact_store(s):
    """Each head as complex numbers: the rotation is a product with e^(i position angle)."""
    rotary, pos = s["case"]["rot"], (s["lens"].double() - 1).clamp(min=0)
    wave = 10000.0 ** (-torch.arange(0, rotary, 2, device="cuda").double() / rotary)
    turn = torch.polar(torch.ones_like(wave), torch.zeros_like(wave)) * torch.exp(1j * pos[:, None] * wave)

    def one(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
        half = rotary // 2
        lead = (torch.complex(x[..., :half].contiguous(), x[..., half:rotary].contiguous()) if s["case"]["pairs"] == "halves"
                else torch.view_as_complex(x[..., :rotary].reshape(*x.shape[:-1], half, 2).contiguous()))
        lead = lead * turn[:, None]
        if s["case"]["pairs"] == "halves":
            x[..., :half], x[..., half:rotary] = lead.real, lead.imag
        else:
            x[..., 0:rotary:2], x[..., 1:rotary:2] = lead.real, lead.imag
        return x

    def stored(cache, x, scale):
        cache = cache.to(torch.float64)
        kept = (s["slots"] >= 0).nonzero()[:, 0]
        x = x[kept] / scale
        cache[s["slots"][kept].long()] = x.clamp(-E4M3_MAX, E4M3_MAX) if s["case"]["cache"] == "e4m3" else x
        return cache

    q = one(s["q"], s["wq"])
    q[s["lens"] <= 0] = 0.0
    return (q, stored(s["k_cache"], one(s["k"], s["wk"]), s["k_scale"]),
            None if s["v"] is None else stored(s["v_cache"], s["v"].double(), s["v_scale"]))


def _exact_attention(s):
    """Request by request and head by head, with each request's keys in their own order."""
    case = s["case"]
    cu, lens, prefix = s["cu"].tolist(), s["seq_lens"].tolist(), s["prefix"].tolist()
    hkv, g, dim = case["hkv"], case["hq"] // case["hkv"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (length, before) in enumerate(zip(lens, prefix)):
        at = torch.arange(length, device="cuda")
        slot = s["table"][s["rows"][b].long()].long()[at // PAGE] * PAGE + at % PAGE
        n = cu[b + 1] - cu[b]
        seen = at[None, :] <= before + torch.arange(n, device="cuda")[:, None]
        if case["block_q"]:
            ids = s["topk"][0, s["cu_blocks"].tolist()[b]:s["cu_blocks"].tolist()[b + 1]]
            listed_ = torch.stack([(ids == j).any(1) for j in range(_blocks(length))], 1)
            seen = seen & listed_.repeat_interleave(case["block_q"], 0)[:n].repeat_interleave(PAGE, 1)[:, :length]
        for h in range(hkv):
            k = s["k_cache"][slot, h].double() * s["k_scale"]
            v = s["v_cache"][slot, h].double() * s["v_scale"]
            q = s["q"][cu[b]:cu[b + 1], h * g:(h + 1) * g].double()
            z = torch.einsum("tgd,kd->tgk", q, k) * s["sm_scale"]
            z = torch.where(seen[:, None], z, -torch.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)  # a row that sees no key is zero
            out[cu[b]:cu[b + 1], h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", p, v)
    return out
