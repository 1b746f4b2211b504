"""The serving-step calls around the paged caches on the GPU, against the
plain 64-bit definitions and the tolerances of serve_ref.py.

Outputs are poisoned before each call, inputs hashed before and after; cache
slots that no request owns hold NaN, so that a value read from one shows.
"""
import math
import random

import numpy as np
import pytest
import torch

import serve_ref as R
from parity import digest, nan_like
from sparse_paged_decode_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BS = 128
I32 = torch.int32
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def spd():
    import sparse_paged_decode_gb300 as m

    return m


def i32(values):
    return torch.tensor(values, dtype=I32, device=DEV)


# ------------------------------------------------------------ slots of a step


def run_assign(spd, new, prefix, rows, free, count, n_pages, bq, table, T, strided=False):
    B = len(new)

    def out(n):
        return nan_like((2 * n + 1,), I32, DEV)[1::2][:n] if strided else nan_like((n,), I32, DEV)

    got = [table.clone(), out(B + 1), out(B + 1), out(B), out(T), out(T), out(T), out(1)]
    ins = (new, prefix, rows, free, count)
    before = digest(*ins)
    spd.paged_assign_slots(*ins, n_pages, BS, bq, *got)
    torch.cuda.synchronize()
    assert digest(*ins) == before, "inputs mutated"
    return got


def check_assign(got, new, prefix, rows, free, count, n_pages, bq, table, T, what):
    ref = R.assign(new, prefix, rows, free, int(count), n_pages, bq, table, T)
    names = ("block_table", "cu_seqlens", "cu_seqblocks_q", "seq_lens", "req_idx", "token_lens", "slots", "free_left")
    for n, g, r in zip(names, got, ref):
        assert np.array_equal(R.ints(g), r), "%s: %s" % (what, n)


ASSIGN = [
    # new, prefix, block_q, NB, T beyond the tokens, free pages short by, strided
    dict(new=[1], prefix=[0], bq=1),
    dict(new=[1, 1, 1], prefix=[127, 128, 129], bq=1),
    dict(new=[0, 5, 0, 300, 0], prefix=[10, 0, 0, 200, 128], bq=64, extra=7),
    dict(new=[0, 0], prefix=[3, 500], bq=4, extra=3),
    dict(new=[], prefix=[], bq=1, extra=4),
    dict(new=[128, 129, 127, 512], prefix=[0, 128, 1, 640], bq=100),
    dict(new=[400, 300, 20], prefix=[0, 100, 1000], bq=16, NB=4),  # past the table's capacity
    dict(new=[700, 300, 400], prefix=[0, 90, 128], bq=3, short=4),  # the free list runs out
    dict(new=[10, 2000000000, 2000000000, 5], prefix=[0, 5, 2147483000, 9], bq=7, extra=-1, NB=8, T=900),  # clipped to T
    dict(new=[-4, 9, 33], prefix=[7, -9, 300], bq=8, extra=2),  # negative counts are 0
    dict(new=[70, 80, 90], prefix=[200, 0, 60], bq=5, extra=9, strided=True),
    dict(new=[70, 80, 90], prefix=[200, 0, 60], bq=5, bad_rows=True),
    dict(new=[70, 80, 400], prefix=[200, 0, 60], bq=5, bad_pages=True),
]


@pytest.mark.parametrize("i", range(len(ASSIGN)))
def test_assign_small(spd, i):
    c = ASSIGN[i]
    new, prefix, NB = c["new"], c["prefix"], c.get("NB", 16)
    B = len(new)
    g = torch.Generator().manual_seed(i)
    rows = torch.randperm(B + 2, generator=g)[:B].to(I32)
    if c.get("bad_rows"):
        rows[0], rows[2] = -1, B + 2
    table = torch.randperm((B + 2) * NB, generator=g).to(I32).view(B + 2, NB)
    n_pages = 1000
    if c.get("bad_pages"):
        table[:, 0], table[:, 1] = -3, n_pages  # cached blocks without a page of the pool
    free = torch.randperm(200, generator=g).to(I32) + 500
    if c.get("bad_pages"):
        free[-2] = n_pages
    grown = sum(max(0, -(-(max(p, 0) + max(n, 0)) // BS) - -(-max(p, 0) // BS)) for n, p in zip(new, prefix))
    count = grown - c["short"] if "short" in c else 200
    T = c.get("T", sum(max(n, 0) for n in new) + c.get("extra", 0))
    args = (i32(new), i32(prefix), rows.to(DEV), free.to(DEV), i32([count]), n_pages, c["bq"], table.to(DEV), T)
    got = run_assign(spd, *args, strided=c.get("strided", False))
    check_assign(got, *args, "case %d" % i)
    # the grown table is the only input that changes: a second call gives the same
    again = run_assign(spd, *args[:7], got[0], T)
    check_assign(again, *args, "case %d again" % i)


@pytest.mark.parametrize("B,T,seed", [(64, 500, 1), (513, 5000, 2), (2048, 66000, 3), (8192, 20000, 4), (8192, 0, 5)])
def test_assign_large(spd, B, T, seed):
    r = random.Random(seed)
    new = [r.choice((0, 1, 1, 4, 16, r.randint(0, 2 * T // B))) for _ in range(B)]
    prefix = [r.randint(0, 1200) for _ in range(B)]
    NB = 24
    g = torch.Generator().manual_seed(seed)
    rows = torch.randperm(B, generator=g).to(I32)
    table = torch.randint(0, 1 << 20, (B, NB), generator=g).to(I32)
    free = (torch.randperm(4 * B, generator=g) + (1 << 20)).to(I32)
    args = (i32(new), i32(prefix), rows.to(DEV), free.to(DEV), i32([3 * B]), 1 << 23, 16, table.to(DEV), T)
    check_assign(run_assign(spd, *args), *args, "B=%d" % B)


# ------------------------------------------------- norm, rotation and store


def store_inputs(T, Hq, Hkv, D, Rd, M, dt, cache, seed, values=True, weights=BF16, pool=None):
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dt).to(DEV)
    pool = pool or (-(-T // BS) + 2)
    angle = torch.rand((M, Rd // 2), generator=g, dtype=torch.float64) * 6.3
    s = dict(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:] if values else None,
             wq=None if weights is None else (1 + 0.2 * torch.randn(D, generator=g)).to(weights).to(DEV),
             wk=None if weights is None else (1 + 0.2 * torch.randn(D, generator=g)).to(weights).to(DEV),
             cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV),
             lens=torch.randint(1, M + 1, (T,), generator=g).to(I32),
             slots=torch.randperm(pool * BS, generator=g)[:T].to(I32))
    s["kc"] = (torch.randn((pool * BS, Hkv, D), generator=g)).to(cache).to(DEV)
    s["vc"] = (torch.randn((pool * BS, Hkv, D), generator=g)).to(cache).to(DEV) if values else None
    return s


def run_store(spd, s, out_dt, eps=1e-6, interleaved=False, ks=1.0, vs=1.0, out=None):
    kc0, vc0 = s["kc"].clone(), s["vc"].clone() if s["vc"] is not None else None
    out = nan_like(s["q"].shape, out_dt, DEV) if out is None else out
    lens, slots = s["lens"].to(DEV), s["slots"].to(DEV)
    ins = (s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos_sin"], lens, slots)
    before = digest(*ins)
    spd.paged_norm_rope_store(*ins, out, s["kc"], s["vc"], eps, interleaved, BS, ks, vs)
    torch.cuda.synchronize()
    assert digest(*ins) == before, "inputs mutated"
    # values
    lens, slots = R.ints(s["lens"]), R.ints(s["slots"])
    M, n_slots = s["cos_sin"].shape[0], s["kc"].shape[0]
    ref, mag = R.head_rows(s["q"], s["wq"], s["cos_sin"], lens, eps, interleaved)
    R.check_kept(out, ref, mag, out_dt, "q_out")
    kept = [t for t in range(len(lens)) if 1 <= lens[t] <= M and 0 <= slots[t] < n_slots]
    ref, mag = R.head_rows(s["k"], s["wk"], s["cos_sin"], lens, eps, interleaved)
    R.check_kept(s["kc"][slots[kept]], ref[kept] / ks, mag[kept] / ks, s["kc"].dtype, "k_cache")
    if s["v"] is not None:
        v = R.f64(s["v"])[kept] / vs
        R.check_kept(s["vc"][slots[kept]], v, np.abs(v), s["vc"].dtype, "v_cache")
    # every other slot as it was
    rest = np.setdiff1d(np.arange(n_slots), slots[kept])
    for now, was in ((s["kc"], kc0), (s["vc"], vc0)):
        if now is not None:
            assert digest(now[rest]) == digest(was[rest]), "a slot that no token names changed"
    return out


STORE = [
    # T, Hq, Hkv, D, Rd, input, cache, output, interleaved, weights, values
    (1, 8, 1, 64, 64, F32, BF16, BF16, False, F32, True),
    (5, 64, 8, 128, 128, BF16, E4M3, BF16, False, BF16, True),
    (33, 64, 8, 128, 64, BF16, BF16, BF16, True, BF16, True),
    (129, 16, 2, 128, 128, F16, E4M3, F16, False, F32, True),
    (17, 6, 3, 96, 32, BF16, E4M3, BF16, False, BF16, True),
    (40, 4, 4, 256, 256, BF16, BF16, BF16, False, BF16, True),
    (9, 3, 1, 7, 6, F32, F32, F32, True, F16, True),
    (9, 2, 1, 1 + 2, 2, BF16, F16, F32, False, None, True),
    (200, 1, 1, 128, 128, BF16, BF16, BF16, False, BF16, False),  # index queries and key
    (64, 4, 1, 128, 128, BF16, E4M3, BF16, False, BF16, False),
    (70, 32, 8, 64, 32, F16, BF16, BF16, True, F16, True),
    (31, 7, 7, 80, 80, BF16, E4M3, F32, True, BF16, True),
]


@pytest.mark.parametrize("policy", [0, 1])
@pytest.mark.parametrize("i", range(len(STORE)))
def test_store_small(spd, i, policy):
    T, Hq, Hkv, D, Rd, dt, cache, out_dt, inter, weights, values = STORE[i]
    s = store_inputs(T, Hq, Hkv, D, Rd, 300, dt, cache, 40 + i, values, weights)
    # padding rows: no position, a position behind the table, no slot, a slot behind the pool
    for t, (n, at) in zip(range(1, T, 3), ((0, 5), (301, 6), (7, -1), (9, s["kc"].shape[0]), (-5, -5))):
        s["lens"][t], s["slots"][t] = n, (at if at < 0 or at >= s["kc"].shape[0] else s["slots"][t])
    old = spd.set_kernel_policy(6, policy)
    try:
        ks, vs = (0.013, 0.02) if cache == E4M3 else (1.0, 1.0)
        run_store(spd, s, out_dt, interleaved=inter, ks=ks, vs=vs)
    finally:
        spd.set_kernel_policy(6, old)


@pytest.mark.parametrize("policy", [0, 1])
def test_store_saturates_and_keeps_nan(spd, policy):
    s = store_inputs(40, 8, 2, 128, 128, 64, BF16, E4M3, 3)
    s["v"][0] = 1000.0
    s["v"][1, 0, 3] = float("nan")
    s["v"][2] = float("inf")
    s["k"][3] = 0.0  # a zero row stays zero (eps > 0)
    old = spd.set_kernel_policy(6, policy)
    try:
        run_store(spd, s, BF16, ks=0.001, vs=0.5)
    finally:
        spd.set_kernel_policy(6, old)


@pytest.mark.parametrize("policy", [0, 1])
@pytest.mark.parametrize("kind", ["odd_offset", "transposed", "interleaved_caches", "broadcast_weight", "strided_out"])
def test_store_strides(spd, kind, policy):
    T, Hq, Hkv, D = 37, 8, 2, 128
    s = store_inputs(T, Hq, Hkv, D, 128, 90, BF16, BF16, 9)
    out = None
    if kind == "odd_offset":  # rows that start off any vector boundary
        wide = torch.randn((T, Hq, D + 3), device=DEV).to(BF16)
        s["q"] = wide[:, :, 1:D + 1]
    elif kind == "transposed":
        s["k"] = s["k"].transpose(0, 1).contiguous().transpose(0, 1)
        s["q"] = s["q"].transpose(1, 2).contiguous().transpose(1, 2)
    elif kind == "interleaved_caches":  # K and V of a slot side by side in one allocation
        both = torch.randn((4 * BS, 2, Hkv, D), device=DEV).to(BF16)
        s["kc"], s["vc"] = both[:, 0], both[:, 1]
        s["slots"] = torch.randperm(4 * BS)[:T].to(I32)
    elif kind == "broadcast_weight":
        s["wq"] = torch.full((1,), 1.5, device=DEV).expand(D)
    else:
        out = nan_like((T, Hq, 2 * D), BF16, DEV)[:, :, ::2]
    old = spd.set_kernel_policy(6, policy)
    try:
        if kind == "interleaved_caches":
            kc, vc = s["kc"], s["vc"]
            run_store(spd, s, BF16)
            assert s["kc"] is kc and s["vc"] is vc
        else:
            run_store(spd, s, BF16, out=out)
    finally:
        spd.set_kernel_policy(6, old)


# --------------------------------------------------------- prefill attention


def chunk_inputs(chunks, prefix, Hq, Hkv, D, q_dt, cache, seed, NB=16, seq_lens=None, spare_rows=2, bq=0, topk=0,
                 per_head=False, q_scale=1.0, nan_pool=True):
    g = torch.Generator().manual_seed(seed)
    B = len(chunks)
    whole = [c + p for c, p in zip(chunks, prefix)]
    need = [max(1, -(-n // BS)) for n in whole]
    P = sum(need) + 5
    table, owned = W._pages_for(whole + [0] * spare_rows, P + spare_rows, NB, g)
    P = P + spare_rows
    perm = torch.randperm(B + spare_rows, generator=g)
    rows = torch.argsort(perm)[:B].to(I32)
    table = table[perm].contiguous()
    cu = np.concatenate(([0], np.cumsum(chunks))).tolist()
    s = dict(q=(q_scale * torch.randn((cu[-1], Hq, D), generator=g)).to(q_dt), table=table, rows=rows, cu=cu,
             prefix=list(prefix), seq_lens=whole if seq_lens is None else list(seq_lens), sm=D ** -0.5, bq=bq, P=P, whole=whole,
             owned=owned)
    slots = torch.cat([W._request_slots(o, n) for o, n in zip(owned[:B], whole)]) if sum(whole) else torch.zeros(0, dtype=torch.int64)
    for name in ("k", "v"):
        vals = torch.randn((len(slots), Hkv, D), generator=g)
        if cache == E4M3:
            codes, scale = W._to_e4m3(vals)
            c = torch.full((P * BS, Hkv, D), 0x7F if nan_pool else 0, dtype=torch.uint8)
            c[slots] = codes.view(torch.uint8)
            s[name + "c"], s[name + "s"] = c.view(E4M3), scale
        else:
            c = torch.full((P * BS, Hkv, D), float("nan") if nan_pool else 0.0, dtype=BF16)
            c[slots] = vals.to(BF16)
            s[name + "c"], s[name + "s"] = c, 1.0
    if bq:
        cub = np.concatenate(([0], np.cumsum([-(-c // bq) for c in chunks]))).tolist()
        heads = Hkv if per_head else 1
        pick = torch.full((heads, max(cub[-1], 1), topk), -1, dtype=I32)
        for h in range(heads):
            for b in range(B):
                for i in range(cub[b + 1] - cub[b]):
                    n = -(-min(prefix[b] + i * bq + 1, whole[b]) // BS)
                    ids = torch.randperm(max(n, 1), generator=g)[:topk]
                    pick[h, cub[b] + i, :len(ids)] = ids.to(I32)
                    pick[h, cub[b] + i, 0] = n - 1  # the block of the tokens themselves
        s["topk"], s["cub"] = (pick if per_head else pick.expand(Hkv, -1, -1)), cub
    return s


def run_chunk(spd, s, out=None, check=True, status=True, what="", q=None):
    q = (s["q"] if q is None else q).to(DEV)
    dev = {n: i32(s[n]) for n in ("cu", "prefix", "seq_lens")}
    kc, vc, table, rows = (s[n].to(DEV) for n in ("kc", "vc", "table", "rows"))
    Hkv, (T, Hq, D) = kc.shape[1], q.shape
    out = nan_like(q.shape, BF16, DEV) if out is None else out
    n_rows = s["topk"].shape[1] if s["bq"] else 0
    size = spd.prefill_attention_workspace_bytes(T, Hq, Hkv, D, len(rows), table.shape[1], n_rows)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    ins = [q, kc, vc, table, rows, dev["cu"], dev["seq_lens"], dev["prefix"]]
    more = []
    if s["bq"]:
        topk = s["topk"][:1].to(DEV).expand(Hkv, -1, -1) if s["topk"].stride(0) == 0 else s["topk"].to(DEV)
        more = [topk, s["bq"], i32(s["cub"])]
    scales = (s["sm"], BS, s["ks"], s["vs"])
    before = digest(*ins)
    if s["bq"]:
        spd.paged_sparse_prefill_attention(*ins, *more, out, *scales, ws)
    else:
        spd.paged_prefill_attention(*ins, out, *scales, ws)
    torch.cuda.synchronize()
    assert digest(*ins) == before, "inputs mutated"
    if status:
        assert spd.workspace_status(ws) == 0, "a wait timed out"
    if check:
        ref, A = R.attention(q, s["kc"], s["vc"], s["table"], s["rows"], torch.tensor(s["cu"]), torch.tensor(s["seq_lens"]),
                             torch.tensor(s["prefix"]), s["sm"], s["ks"], s["vs"], s.get("topk"), s["bq"],
                             None if not s["bq"] else torch.tensor(s["cub"]))
        R.check_attention(out, ref, A, what)
    return out


class policy:
    def __init__(self, spd, value):
        self.spd, self.value = spd, value

    def __enter__(self):
        self.old = self.spd.set_kernel_policy(5, self.value)

    def __exit__(self, *exc):
        self.spd.set_kernel_policy(5, self.old)


CHUNKS = {
    "one_token": ([1], [0]),
    "one_token_late": ([1], [700]),
    "page_edge": ([1, 2, 128, 129], [127, 127, 128, 0]),
    "ragged": ([70, 5, 130, 1, 33], [300, 0, 1000, 77, 128]),
    "empty_chunks": ([0, 9, 0, 40, 0], [5, 250, 0, 0, 640]),
    "long_over_short": ([300], [0]),
    "short_over_long": ([3, 17], [1900, 1500]),
}


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("name", CHUNKS)
def test_prefill_attention_small(spd, name, cache, pol):
    chunks, prefix = CHUNKS[name]
    with policy(spd, pol):
        run_chunk(spd, chunk_inputs(chunks, prefix, 16, 2, 128, BF16, cache, 70), what=name)


HEADS = [(8, 1, 64, BF16), (64, 8, 128, BF16), (3, 3, 128, BF16), (6, 2, 128, BF16), (14, 2, 128, BF16), (16, 1, 128, BF16),
         (8, 2, 64, BF16), (4, 2, 96, BF16), (2, 1, 256, BF16), (8, 2, 7, BF16), (8, 2, 128, F32), (8, 2, 128, F16), (8, 2, 64, F16)]


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d_%d_%d_%s" % (h[0], h[1], h[2], str(h[3])[6:]))
def test_prefill_attention_heads(spd, heads, cache, pol):
    Hq, Hkv, D, dt = heads
    with policy(spd, pol):
        run_chunk(spd, chunk_inputs([40, 7, 150], [200, 0, 130], Hq, Hkv, D, dt, cache, 71), what=str(heads))


SPARSE = [
    # chunks, prefix, block_q, topk, per head
    ([70, 5, 130, 1, 33], [300, 0, 1000, 77, 128], 16, 4, False),
    ([70, 5, 130, 1, 33], [300, 0, 1000, 77, 128], 1, 3, True),
    ([200, 64, 33], [1500, 20, 900], 64, 5, True),
    ([200, 64, 33], [1500, 20, 900], 100, 40, False),  # wider than the visible blocks
    ([128, 256], [0, 640], 128, 1, False),
    ([3, 0, 50], [1000, 3, 1900], 7, 8, True),
]


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("i", range(len(SPARSE)))
def test_sparse_prefill_attention(spd, i, cache, pol):
    chunks, prefix, bq, topk, per_head = SPARSE[i]
    s = chunk_inputs(chunks, prefix, 16, 2, 128, BF16, cache, 72 + i, bq=bq, topk=topk, per_head=per_head)
    # repeated, negative and too large ids select nothing more
    if topk > 2:
        pick = s["topk"][:1].clone() if not per_head else s["topk"]
        pick[:, ::2, 1] = pick[:, ::2, 0]
        pick[:, 1::3, 2] = 4000
        pick[:, 1::4, 1] = -7
        s["topk"] = pick if per_head else pick.expand(2, -1, -1)
    with policy(spd, pol):
        run_chunk(spd, s, what=str(SPARSE[i]))


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("bq", [0, 16, 64], ids=["dense", "bq16", "bq64"])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_prefill_attention_metadata(spd, cache, bq, pol):
    """Rows outside the table, pages outside the pool, seq_lens short of the
    chunk, past the table and zero, negative prefixes, tokens that no sequence
    owns in front of, between and behind the chunks."""
    chunks, prefix = [60, 30, 100, 20, 90, 10], [500, 0, 300, 100, 200, 640]
    s = chunk_inputs(chunks, prefix, 16, 2, 128, BF16, cache, 90 + bq, bq=bq, topk=4)
    s["rows"][1], s["rows"][3] = -1, s["table"].shape[0]
    s["table"][s["rows"][0], 2] = -1
    s["table"][s["rows"][2], 0] = s["P"]
    s["table"][s["rows"][2], 3] = 1 << 29
    s["seq_lens"][2], s["seq_lens"][4], s["seq_lens"][5] = 350, 0, 1 << 30
    s["prefix"][4] = -20
    s["cu"] = [c + 5 for c in s["cu"]]  # five unowned tokens in front, seven behind
    s["q"] = torch.randn((s["cu"][-1] + 7, 16, 128)).to(BF16)
    if bq:
        s["cub"][-1] -= 1  # the last query block has no row of its own
    with policy(spd, pol):
        # the last request runs behind its keys: those slots are NaN, so it is held to the keys that it owns
        s["seq_lens"][5] = s["whole"][5]
        run_chunk(spd, s, what="metadata")


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("bq", [0, 4], ids=["dense", "bq4"])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_unread_keys_never_reach_a_row(spd, cache, bq, bad, pol):
    """A later key of the chunk itself that is not finite: the tokens in front
    of it (and those that did not select its block) are what they were."""
    if cache == E4M3 and bad != bad:
        code = 0x7F
    elif cache == E4M3:
        pytest.skip("E4M3 has no infinity")
    s = chunk_inputs([90, 40], [250, 0], 16, 2, 128, BF16, cache, 95, bq=bq, topk=2)
    with policy(spd, pol):
        clean = run_chunk(spd, s, what="clean")
        at = 250 + 61  # position of the spoilt key: token 61 of the first chunk reads it first
        slot = int(s["owned"][0][at // BS]) * BS + at % BS
        for name in ("kc", "vc"):
            if cache == E4M3:
                s[name].view(torch.uint8)[slot, :, ::3] = code
            else:
                s[name][slot, :, ::3] = bad
        got = run_chunk(spd, s, check=False)
    reads = torch.zeros(130, dtype=torch.bool)
    for t in range(61, 90):
        reads[t] = bq == 0 or (at // BS) in s["topk"][0, s["cub"][0] + t // bq].tolist()
    assert reads.any()
    # a NaN logit or a non-finite value shows in the rows that read it ...
    assert not torch.isfinite(got.float().cpu()[reads][..., ::3]).any()
    # ... and in no other: bit for bit the same
    assert torch.equal(got.cpu()[~reads].view(torch.int16), clean.cpu()[~reads].view(torch.int16))


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_prefill_attention_large_logits_and_strides(spd, cache, pol):
    s = chunk_inputs([50, 130], [400, 100], 16, 2, 128, BF16, cache, 96, q_scale=6.0)
    with policy(spd, pol):
        run_chunk(spd, s, what="large logits")
        s["sm"] = -s["sm"]
        run_chunk(spd, s, what="negative scale")
        s["sm"] = 0.0
        run_chunk(spd, s, what="zero scale")
        s["sm"] = 128 ** -0.5
        wide = torch.randn((180, 2 * 16, 128)).to(BF16).to(DEV)
        out = nan_like((180, 16, 256), BF16, DEV)
        run_chunk(spd, s, out=out[:, :, 1:129], q=wide[:, ::2], what="strides")
        odd = torch.randn((180, 16, 131)).to(BF16).to(DEV)[:, :, 1:129]
        run_chunk(spd, s, q=odd, what="odd rows")
        rest = out.clone()
        rest[:, :, 1:129] = float("nan")
        assert torch.isnan(rest.float()).all(), "cells beside the output were written"


@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("bq", [0, 64], ids=["dense", "bq64"])
def test_prefill_attention_graph_replay(spd, bq, cache):
    """A captured call replays with new lengths, tables, selections and values
    at the same addresses, while a call on another stream uses a workspace of
    its own."""
    a = chunk_inputs([100, 60, 40], [900, 0, 300], 16, 2, 128, BF16, cache, 97, bq=bq, topk=4)
    b = chunk_inputs([20, 150, 30], [1200, 130, 0], 16, 2, 128, BF16, cache, 98, bq=bq, topk=4)
    if bq:  # as many selection rows in both
        rows = max(a["topk"].shape[1], b["topk"].shape[1])
        for s in (a, b):
            pad = torch.full((1, rows, 4), -1, dtype=I32)
            pad[:, :s["topk"].shape[1]] = s["topk"][:1]
            s["topk"] = pad.expand(2, -1, -1)
    pool = max(a["P"], b["P"])
    names = ["q", "kc", "vc", "table", "rows", "cu", "seq_lens", "prefix"] + (["topk", "cub"] if bq else [])

    def on_device(s):
        d = {n: (s[n] if torch.is_tensor(s[n]) else torch.tensor(s[n], dtype=I32)) for n in names}
        for n in ("kc", "vc"):
            full = torch.zeros((pool * BS,) + tuple(d[n].shape[1:]), dtype=d[n].dtype)
            full.view(torch.uint8)[:d[n].shape[0]] = d[n].view(torch.uint8)
            d[n] = full
        return {n: (d[n][:1] if n == "topk" else d[n]).contiguous().to(DEV) for n in names}

    def call(d, s, out, ws):
        head = [d[n] for n in names[:8]]
        scales = (a["sm"], BS, a["ks"], a["vs"], ws)
        if bq:
            spd.paged_sparse_prefill_attention(*head, d["topk"].expand(2, -1, -1), bq, d["cub"], out, *scales)
        else:
            spd.paged_prefill_attention(*head, out, *scales)

    b["ks"], b["vs"] = a["ks"], a["vs"]
    d, e = on_device(a), on_device(b)
    size = spd.prefill_attention_workspace_bytes(200, 16, 2, 128, 3, 16, d["topk"].shape[1] if bq else 0)
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2))
    out, out2 = (nan_like((200, 16, 128), BF16, DEV) for _ in range(2))
    eager = [run_chunk(spd, s, what="eager") for s in (a, b)]
    call(d, a, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        call(d, a, out, ws)
    for s, src in ((a, d), (b, e), (a, None)):
        if src is None:
            src = on_device(a)
        for n in names:
            d[n].copy_(src[n]) if s is not a or src is not d else None
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            call(e, b, out2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager[0 if s is a else 1].view(torch.int16))
        assert torch.equal(out2.view(torch.int16), eager[1].view(torch.int16))


@pytest.mark.parametrize("kind", ["e4m3", "e4m3_f16", "bf16", "e4m3_d64"])
@pytest.mark.parametrize("bq", [0, 16], ids=["dense", "bq16"])
def test_prefill_attention_many_units(spd, bq, kind):
    """Several units to a CTA, in turn with one tile of query rows and with
    two, without pages and with many, split and whole."""
    r = random.Random(11)
    chunks = [r.choice((1, 3, 9, 16, 17, 30, 33, 60)) for _ in range(60)]
    prefix = [r.choice((0, 0, 5, 130, 700, 1300)) for _ in chunks]
    s = chunk_inputs(chunks, prefix, 64, 8, 64 if kind == "e4m3_d64" else 128, F16 if kind == "e4m3_f16" else BF16,
                     BF16 if kind == "bf16" else E4M3, 101, bq=bq, topk=3)
    for b in (3, 17, 40):  # requests without a page-table row: their units have no pages
        s["rows"][b] = -1
    run_chunk(spd, s, what="many units")


def test_prefill_attention_long_splits(spd):
    """Few rows over a long cache: the keys are split over many CTAs and joined."""
    for cache in (E4M3, BF16):
        for chunks, prefix in (([16, 1], [15000, 9000]), ([33], [16000])):
            s = chunk_inputs(chunks, prefix, 64, 8, 128, BF16, cache, 99, NB=128)
            outs = [run_chunk(spd, s, what="long %s" % chunks) for _ in range(1)]
            outs.append(run_chunk(spd, s, check=False))
            assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16)), "two runs differ"


def test_far_pages_of_a_large_cache(spd):
    """Offsets past 2^31 elements: pages at the end of a cache of 2.6 G elements."""
    Hkv, D, P = 8, 128, 20000
    cache = torch.zeros((P * BS, Hkv, D), dtype=torch.uint8, device=DEV)
    s = chunk_inputs([40], [300], 64, Hkv, D, BF16, E4M3, 100)
    far = [P - 1, P - 7, P - 3]
    small = s["owned"][0].tolist()
    kc, vc = cache.view(E4M3), cache.clone().view(E4M3)
    for f, p in zip(far, small):
        for big, name in ((kc, "kc"), (vc, "vc")):
            big.view(torch.uint8)[f * BS:(f + 1) * BS] = s[name].view(torch.uint8)[p * BS:(p + 1) * BS].to(DEV)
    ref = run_chunk(spd, s, what="near")
    table = s["table"].clone()
    table[s["rows"][0], :3] = torch.tensor(far, dtype=I32)
    out = nan_like(s["q"].shape, BF16, DEV)
    ws = torch.empty(spd.prefill_attention_workspace_bytes(40, 64, Hkv, D, 1, 16, 0), dtype=torch.uint8, device=DEV)
    spd.paged_prefill_attention(s["q"].to(DEV), kc, vc, table.to(DEV), s["rows"].to(DEV), i32(s["cu"]), i32(s["seq_lens"]),
                                i32(s["prefix"]), out, s["sm"], BS, s["ks"], s["vs"], ws)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    # and a token stored there
    st = store_inputs(3, 4, Hkv, D, 128, 64, BF16, E4M3, 5, values=False)
    st["slots"] = torch.tensor([P * BS - 1, P * BS - 300, 5], dtype=I32)
    keep = st["kc"]
    st["kc"] = kc
    q_out = nan_like(st["q"].shape, BF16, DEV)
    spd.paged_norm_rope_store(st["q"], st["k"], None, st["wq"], st["wk"], st["cos_sin"], st["lens"].to(DEV),
                              st["slots"].to(DEV), q_out, kc, None, 1e-6, False, BS, 0.02, 1.0)
    near = keep
    spd.paged_norm_rope_store(st["q"], st["k"], None, st["wq"], st["wk"], st["cos_sin"], st["lens"].to(DEV),
                              i32([1, 2, 3]), q_out, near, None, 1e-6, False, BS, 0.02, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(torch.uint8)[st["slots"].long().to(DEV)], near.view(torch.uint8)[1:4])


def test_both_ways_of_marshalling(spd, monkeypatch):
    """The compiled module and the Python descriptors pass the same call."""
    from sparse_paged_decode_gb300 import binding

    if binding._fast is None:
        pytest.skip("the marshalling module is not built here")
    args = (i32([70, 80, 90]), i32([200, 0, 60]), i32([2, 0, 1]), i32(list(range(30))), i32([30]), 64, 5,
            torch.arange(64, dtype=I32, device=DEV).view(4, 16), 240)
    st = store_inputs(30, 8, 2, 128, 64, 50, BF16, E4M3, 6)
    ch = chunk_inputs([40, 7], [200, 0], 8, 2, 128, BF16, E4M3, 7, bq=16, topk=2)
    got = []
    for way in (binding._fast, None):
        monkeypatch.setattr(binding, "_fast", way)
        s = dict(st, kc=st["kc"].clone(), vc=st["vc"].clone())
        got.append([*run_assign(spd, *args, strided=True), run_store(spd, s, BF16, ks=0.1, vs=0.1), s["kc"].view(torch.uint8),
                    s["vc"].view(torch.uint8), run_chunk(spd, ch), run_chunk(spd, dict(ch, bq=0, topk=None))])
        with pytest.raises(binding.SpdError):
            spd.paged_assign_slots(*args[:5], -1, BS, 5, *got[-1][:8])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        spd.paged_assign_slots(*args[:5], 64, BS, 5, *got[-1][:8], stream=side)
        side.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------ the whole step


@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_serving_steps(spd, cache):
    """Two steps of a serving loop: slots assigned, q, k, v and the index
    tensors normalised, rotated and stored, blocks selected, attention over
    them, and the dense call over the same caches; each call is held to its
    definition on the inputs that the call before it left."""
    torch.manual_seed(7)
    B, Hq, Hkv, D, NB, bq, K = 3, 16, 2, 128, 12, 16, 4
    pool, M = 40, NB * BS
    free = torch.randperm(pool, device=DEV).to(I32)
    count = i32([pool])
    table = torch.full((B, NB), -1, dtype=I32, device=DEV)
    rows = i32([2, 0, 1])
    kc, vc = (torch.full((pool * BS, Hkv, D), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3) if cache == E4M3 else
              torch.full((pool * BS, Hkv, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    kic = torch.full((pool * BS, 1, D), float("nan"), dtype=BF16, device=DEV)
    angle = torch.arange(M, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV)
    w = [(1 + 0.1 * torch.randn(D, device=DEV)).to(BF16) for _ in range(4)]
    ks = vs = 0.02 if cache == E4M3 else 1.0
    prefix = [0, 0, 0]
    for step, new in enumerate(([500, 40, 300], [30, 400, 1])):
        T = sum(new)
        out = [nan_like((n,), I32, DEV) for n in (B + 1, B + 1, B, T, T, T, 1)]
        cu, cub, sl, req, lens, slots, left = out
        before = table.clone()
        spd.paged_assign_slots(i32(new), i32(prefix), rows, free, count, pool, BS, bq, table, *out)
        torch.cuda.synchronize()
        check_assign([table] + out, i32(new), i32(prefix), rows, free, count, pool, bq, before, T, "step %d" % step)
        count = left
        x = torch.randn((T, Hq + 2 * Hkv + 3, D), device=DEV).to(BF16)
        q, qi = nan_like((T, Hq, D), BF16, DEV), nan_like((T, 2, D), BF16, DEV)
        st = dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:Hq + 2 * Hkv], wq=w[0], wk=w[1], cos_sin=cos_sin,
                  lens=lens, slots=slots, kc=kc, vc=vc)
        run_store(spd, st, BF16, ks=ks, vs=vs, out=q)
        ix = dict(q=x[:, Hq + 2 * Hkv:Hq + 2 * Hkv + 2], k=x[:, -1:], v=None, wq=w[2], wk=w[3], cos_sin=cos_sin, lens=lens,
                  slots=slots, kc=kic, vc=None)
        run_store(spd, ix, BF16, out=qi)
        n_rows = int(cub[-1])
        topk = nan_like((2, n_rows, K), I32, DEV)
        pws = torch.empty(spd.prefill_workspace_bytes(T, 2, NB), dtype=torch.uint8, device=DEV)
        spd.msa_prefill_block_score(qi, kic, table, rows, cu, sl, i32(prefix), bq, BS, 1, 1, D ** -0.5, cub, topk, pws)
        for sparse in (False, True):
            o = nan_like((T, Hq, D), BF16, DEV)
            ws = torch.empty(spd.prefill_attention_workspace_bytes(T, Hq, Hkv, D, B, NB, n_rows if sparse else 0),
                             dtype=torch.uint8, device=DEV)
            head = (q, kc, vc, table, rows, cu, sl, i32(prefix))
            if sparse:
                spd.paged_sparse_prefill_attention(*head, topk, bq, cub, o, D ** -0.5, BS, ks, vs, ws)
            else:
                spd.paged_prefill_attention(*head, o, D ** -0.5, BS, ks, vs, ws)
            torch.cuda.synchronize()
            ref, A = R.attention(q, kc, vc, table, rows, cu, sl, torch.tensor(prefix), D ** -0.5, ks, vs,
                                 topk if sparse else None, bq, cub)
            R.check_attention(o, ref, A, "step %d %s" % (step, "sparse" if sparse else "dense"))
        prefix = R.ints(sl).tolist()


# ------------------------------------------------ what is read and not finite


def held(spd, s, what):
    """A run whose rows are NaN exactly where the 64-bit definition's are, and
    within the usual bounds elsewhere."""
    got = run_chunk(spd, s, check=False).float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        ref, A = R.attention(s["q"], s["kc"], s["vc"], s["table"], s["rows"], torch.tensor(s["cu"]),
                             torch.tensor(s["seq_lens"]), torch.tensor(s["prefix"]), s["sm"], s["ks"], s["vs"], s.get("topk"),
                             s["bq"], None if not s["bq"] else torch.tensor(s["cub"]))
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what + ": NaN pattern"
    R.check_attention(torch.from_numpy(np.where(nan, 0.0, got)), np.where(nan, 0.0, ref), np.where(nan, 0.0, A), what)
    return nan


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("kind", ["e4m3", "e4m3_f16", "e4m3_d64", "bf16"])
@pytest.mark.parametrize("bq", [0, 8], ids=["dense", "bq8"])
def test_infinite_queries(spd, bq, kind, pol):
    """A query row with an infinity has no finite softmax: NaN, and nothing
    in its neighbours.  One that reads no key stays zero."""
    D = 64 if kind == "e4m3_d64" else 128
    s = chunk_inputs([30, 12, 5], [300, 0, 40], 16, 2, D, F16 if kind == "e4m3_f16" else BF16,
                     BF16 if kind == "bf16" else E4M3, 120, bq=bq, topk=2)
    s["rows"][2] = -1
    inf = float("inf")
    s["q"][3, 5, 7], s["q"][17, 0, 0], s["q"][33, 15, D - 1] = inf, -inf, inf
    s["q"][20, 9, ::2] = -inf
    s["q"][44, 3, 1] = inf  # of the request that reads nothing
    with policy(spd, pol):
        nan = held(spd, s, "infinite queries")
    rows = nan.any(-1)
    assert rows.sum() == 4 and rows[3, 5] and rows[17, 0] and rows[33, 15] and rows[20, 9]


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("bq", [0, 8], ids=["dense", "bq8"])
@pytest.mark.parametrize("chunk", [9, 40])
def test_keys_of_minus_infinity(spd, chunk, bq, pol):
    """Logits of -inf weigh nothing beside others, wherever the keys are cut
    into steps, pages, tiles and pieces; a row with no others is NaN."""
    prefix = 1500
    s = chunk_inputs([chunk, chunk], [prefix, 260], 16, 2, 128, BF16, BF16, 121, bq=bq, topk=4)
    s["q"] = s["q"].abs() + 0.125  # times -inf: -inf, never NaN
    own = [o.tolist() for o in s["owned"][:2]]
    for b, blocks in ((0, (0, 1, 2, 5, 6, 11)), (1, (0, 1))):
        for kb in blocks:
            s["kc"][own[b][kb] * BS:(own[b][kb] + 1) * BS, :, 3] = -float("inf")
    at = own[1][2] * BS  # the second request's third block up to its fifth new token: rows without another key
    s["kc"][at:at + 4 + 5, 1, 3] = -float("inf")
    with policy(spd, pol):
        nan = held(spd, s, "keys of -inf")
    if not bq:  # selections may hold nothing but such keys, too
        assert not nan[:chunk].any() and not nan[:, :8].any()
        assert nan[chunk:chunk + 5, 8:].all() and not nan[chunk + 5:].any()


@pytest.mark.parametrize("bq", [0, 1], ids=["dense", "bq1"])
@pytest.mark.parametrize("B", [600, 1500, 8192])
def test_prefill_attention_many_sequences(spd, B, bq):
    """More sequences than are ranked by length, and than have their pairs in
    shared memory, up to the most that a call takes."""
    r = random.Random(B)
    chunks = [r.choice((0, 1, 1, 1, 2)) for _ in range(B)]
    prefix = [r.choice((0, 3, 60, 127)) for _ in chunks]
    s = chunk_inputs(chunks, prefix, 2, 1, 64, BF16, BF16, 122, NB=2, bq=bq, topk=2)
    run_chunk(spd, s, what="%d sequences" % B)


def test_workspace_must_be_one_run(spd, monkeypatch):
    from sparse_paged_decode_gb300 import binding

    s = chunk_inputs([4], [10], 16, 2, 128, BF16, BF16, 123)
    args = [s[n].to(DEV) for n in ("q", "kc", "vc", "table", "rows")] + [i32(s[n]) for n in ("cu", "seq_lens", "prefix")]
    out = nan_like(s["q"].shape, BF16, DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV).expand(1 << 20, 256)
    for way in {binding._fast, None}:
        monkeypatch.setattr(binding, "_fast", way)
        with pytest.raises(ValueError):
            spd.paged_prefill_attention(*args, out, s["sm"], BS, 1.0, 1.0, ws)
    torch.cuda.synchronize()
    assert torch.isnan(out.float()).all(), "a refused call wrote its output"


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_tokens_without_a_sequence(spd, cache, pol):
    """A padded batch with no sequence in it, and one whose selection has no
    rows: zeros, and nothing beside them."""
    q = torch.randn((37, 16, 128), device=DEV).to(BF16)
    kv = torch.full((2 * BS, 2, 128), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3)
    if cache == BF16:
        kv = torch.full((2 * BS, 2, 128), float("nan"), device=DEV).to(BF16)
    none, table = i32([]), i32([[0, 1], [1, 0]])
    with policy(spd, pol):
        for rows, cu, lens, cub in ((none, i32([0]), none, i32([0])), (i32([1]), i32([3, 30]), i32([100]), i32([0, 0]))):
            out = nan_like((39, 16, 128), BF16, DEV)
            size = spd.prefill_attention_workspace_bytes(37, 16, 2, 128, len(rows), 2, 0)
            ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
            topk = torch.empty((2, 0, 3), dtype=I32, device=DEV)
            spd.paged_sparse_prefill_attention(q, kv, kv, table, rows, cu, lens, lens, topk, 4, cub, out[1:38], 0.1, BS,
                                               1.0, 1.0, ws)
            torch.cuda.synchronize()
            assert spd.workspace_status(ws) == 0
            assert not out[1:38].any() and torch.isnan(out[::38].float()).all()
            if len(rows) == 0:
                out.fill_(float("nan"))
                spd.paged_prefill_attention(q, kv, kv, table, rows, cu, lens, lens, out[1:38], 0.1, BS, 1.0, 1.0, ws)
                torch.cuda.synchronize()
                assert not out[1:38].any() and torch.isnan(out[::38].float()).all()


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("kind", ["e4m3", "e4m3_f16", "e4m3_d64", "bf16"])
def test_small_weights_keep_their_bits(spd, kind, pol):
    """One key takes nearly all of the weight and holds zeros: the output is
    the others', 20.5 * 2^-24 of weight each, half a step between two f16
    values if the largest weight is 1."""
    D = 64 if kind == "e4m3_d64" else 128
    s = chunk_inputs([20, 3], [300, 700], 8, 1, D, F16 if kind == "e4m3_f16" else BF16, BF16 if kind == "bf16" else E4M3, 124)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    one = 0x38 if kind != "bf16" else 1.0
    kc, vc = (s[n].view(torch.uint8) if kind != "bf16" else s[n] for n in ("kc", "vc"))
    for o in s["owned"][:2]:
        for page in o.tolist():
            kc[page * BS:(page + 1) * BS] = 0
        kc[int(o[0]) * BS, :, 0] = one
        vc[int(o[0]) * BS] = 0
    s["ks"], s["sm"] = 1.0, float(24 * np.log(2.0) - np.log(20.5))
    with policy(spd, pol):
        run_chunk(spd, s, what="small weights")
