"""Serving-step calls on the GPU at the edges of their range: units of which a
tile takes nothing, heads that end inside a warp, infinities behind a join,
long page tables.  Definitions and tolerances are those of serve_ref.py."""
import numpy as np
import pytest
import torch

import serve_ref as R
from parity import nan_like
from test_serve_gpu import (BF16, BS, DEV, E4M3, F16, I32, check_assign, chunk_inputs, i32, policy, run_assign, run_chunk,
                            run_store, store_inputs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spd():
    import sparse_paged_decode_gb300 as m

    return m


KINDS = ["e4m3", "e4m3_f16", "e4m3_d64", "bf16"]


def kind_of(kind):
    """(head dim, query type, cache type)"""
    return 64 if kind == "e4m3_d64" else 128, F16 if kind == "e4m3_f16" else BF16, BF16 if kind == "bf16" else E4M3


def bits(x):
    return x.view(torch.int16)


# ----------------------------------------------- tiles that take nothing


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("empty", [0, 1], ids=["first_tile", "second_tile"])
def test_units_of_one_page_that_one_tile_takes(spd, kind, empty):
    """Query blocks as long as a tile (16 tokens of 8 heads); in every second
    pair of them one block selects nothing and the other one page, so that a
    unit holds two tiles of queries and one page of which one tile takes
    nothing.  Units with full selections lie between them, several to a CTA."""
    D, q_dt, cache = kind_of(kind)
    chunks, prefix = [640, 480, 96, 320, 64, 33], [300, 0, 900, 1200, 40, 128]
    s = chunk_inputs(chunks, prefix, 64, 8, D, q_dt, cache, 140, bq=16, topk=4)
    pick = s["topk"][:1].clone()
    for b in range(len(chunks)):
        for pair in range(-(-chunks[b] // 32)):
            if pair % 2:
                continue
            rows = [r for r in (s["cub"][b] + 2 * pair, s["cub"][b] + 2 * pair + 1) if r < s["cub"][b + 1]]
            for i, r in enumerate(rows):
                if i == empty:
                    pick[0, r] = -1
                else:
                    pick[0, r, 1:] = -1
    s["topk"] = pick.expand(8, -1, -1)
    first = run_chunk(spd, s, what="one page, one tile")
    for _ in range(3):
        assert torch.equal(bits(run_chunk(spd, s, check=False)), bits(first)), "two runs differ"


# ------------------------------------------- heads that end inside a warp

UNEVEN = [
    # Hq, Hkv, D, values: row groups of one warp with different numbers of rows
    (1, 1, 64, True), (1, 1, 128, True), (2, 2, 64, True), (3, 3, 64, True), (3, 3, 128, True), (5, 5, 64, True),
    (6, 6, 64, True), (10, 5, 64, True), (15, 5, 64, True), (25, 5, 64, True), (17, 17, 128, False), (17, 17, 128, True),
    (33, 11, 128, True), (70, 35, 64, False), (3, 3, 256, True), (100, 50, 256, True),
]


@pytest.mark.parametrize("cache", [E4M3, BF16, F16], ids=["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("shape", UNEVEN, ids=lambda u: "%d_%d_%d_%s" % u)
def test_store_heads_that_end_inside_a_warp(spd, shape, cache):
    Hq, Hkv, D, values = shape
    dt = BF16 if cache != F16 else F16
    for T, Rd, inter in ((1, D, False), (3, D // 2, False), (29, D, True)):
        s = store_inputs(T, Hq, Hkv, D, Rd, 64, dt, cache, 150 + T, values)
        if T > 4:
            s["lens"][2], s["slots"][3] = 0, -1
        ks, vs = (0.013, 0.02) if cache == E4M3 else (1.0, 1.0)
        run_store(spd, s, dt, interleaved=inter, ks=ks, vs=vs)


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("given", ["q", "k"])
@pytest.mark.parametrize("dt,cache,inter", [(F16, F16, False), (F16, F16, True), (BF16, E4M3, True), (F16, E4M3, True),
                                            (BF16, BF16, False)])
def test_store_norm_of_one_of_both(spd, dt, cache, inter, given, pol):
    """Queries with a norm beside keys without one, and the other way round."""
    s = store_inputs(41, 8, 2, 128, 64, 90, dt, cache, 160)
    s["wk" if given == "q" else "wq"] = None
    old = spd.set_kernel_policy(6, pol)
    try:
        run_store(spd, s, dt, interleaved=inter, ks=0.02 if cache == E4M3 else 1.0, vs=0.02 if cache == E4M3 else 1.0)
    finally:
        spd.set_kernel_policy(6, old)


# ------------------------------------------- infinite values that a row reads


def held_with_infinities(spd, s, what):
    """A run whose NaN and infinite cells, signs included, are those of the
    64-bit definition; the finite ones within the usual bounds."""
    got = run_chunk(spd, s, check=False).float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        ref, A = R.attention(s["q"], s["kc"], s["vc"], s["table"], s["rows"], torch.tensor(s["cu"]),
                             torch.tensor(s["seq_lens"]), torch.tensor(s["prefix"]), s["sm"], s["ks"], s["vs"], s.get("topk"),
                             s["bq"], None if not s["bq"] else torch.tensor(s["cub"]))
    odd = ~np.isfinite(ref)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    assert same[odd].all(), "%s: %d of %d cells that are not finite differ" % (what, (~same[odd]).sum(), odd.sum())
    R.check_attention(torch.from_numpy(np.where(odd, 0.0, got)), np.where(odd, 0.0, ref), np.where(odd, 0.0, A), what)
    return odd


def requests_like_it(s, n):
    """The batch of n requests with the pages, lengths and selections of the
    only one in `s`, and queries of their own: so many that none is cut into
    pieces."""
    chunk = s["cu"][1]
    g = torch.Generator().manual_seed(n)
    more = dict(q=torch.randn((n * chunk,) + tuple(s["q"].shape[1:]), generator=g).to(s["q"].dtype), rows=s["rows"][:1].repeat(n),
                cu=[chunk * i for i in range(n + 1)], prefix=s["prefix"] * n, seq_lens=s["seq_lens"] * n)
    if s["bq"]:
        rows = s["cub"][1]
        more.update(topk=s["topk"][:1, :rows].repeat(1, n, 1).expand(s["topk"].shape[0], -1, -1), cub=[rows * i for i in range(n + 1)])
    return dict(s, **more)


@pytest.mark.parametrize("pol", [0, 1])
@pytest.mark.parametrize("n", [1, 200])  # cut into pieces, and whole
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_values_where_the_other_pages_weigh_nothing(spd, D, n, pol):
    """Three tokens, one tile of rows that two tiles work on page by page:
    rows that read an infinite value of one tile's page and nothing of the
    other's."""
    s = chunk_inputs([3], [900], 64, 8, D, BF16, BF16, 170, bq=1, topk=4)
    # blocks 1, 2, 4, 5 are listed: two for each tile, in turn
    s["topk"] = torch.tensor([[[2, 5, -1, -1], [1, 4, -1, -1], [1, 2, 4, 5]]], dtype=I32).expand(8, -1, -1)
    page = s["owned"][0].tolist()
    inf = float("inf")
    s["vc"][page[5] * BS + 9, 0, 3], s["vc"][page[5] * BS + 100, 1, D - 1] = inf, -inf
    s["vc"][page[4] * BS + 1, 0, 33], s["vc"][page[4] * BS + 2, 1, 0] = -inf, inf
    s["vc"][page[2] * BS, 0, 17], s["vc"][page[1] * BS + 127, 0, 17] = inf, -inf  # both: NaN
    with policy(spd, pol):
        odd = held_with_infinities(spd, requests_like_it(s, n), "infinite values")
    odd = odd.reshape(n, 3, 64, D)
    assert odd[:, 0, :8, 3].all() and odd[:, 1, :8, 33].all() and odd[:, 2, :8, 17].all() and not odd[:, 1, :8, 3].any()


@pytest.mark.parametrize("n", [1, 200])
def test_infinite_values_beside_a_weight_of_zero(spd, n):
    """The same with every key read: the first page's logits lie so far below
    the second's that its weight is 0 in 32 bits.  The second page ends inside
    the chunk, so its infinities are looked up."""
    s = requests_like_it(chunk_inputs([3], [200], 64, 8, 128, BF16, BF16, 171), n)
    s["q"] = s["q"].abs() + 0.5
    page = s["owned"][0].tolist()
    s["kc"][page[0] * BS:(page[0] + 1) * BS] = -32.0  # logits below -32 * 128 * 0.5 / sqrt(128) = -181
    s["kc"][page[1] * BS:page[1] * BS + 203 - BS] = 0.0
    s["vc"][page[1] * BS + 3, 0, 5], s["vc"][page[1] * BS + 60, 1, 77] = float("inf"), -float("inf")
    odd = held_with_infinities(spd, s, "weight of zero")
    assert odd[:, :8, 5].all() and odd[:, 8:16, 77].all() and odd.sum() == 2 * 3 * n * 8


# --------------------------------------------------------- long page tables


@pytest.mark.parametrize("kind,pol", [(k, 0) for k in KINDS] + [("e4m3", 1)])
@pytest.mark.parametrize("NB", [129, 1024])
def test_attention_over_long_page_tables(spd, NB, kind, pol):
    """Page tables of up to 1024 blocks: page lists and bitmaps to their last
    word, a request that ends at the table's end and one that ends inside."""
    D, q_dt, cache = kind_of(kind)
    whole, half = NB * BS, NB * BS // 2 - 77
    chunks = [3, 17]
    with policy(spd, pol):
        for bq, topk, per_head in ((0, 0, False), (2, 40, True), (16, 600, False)):
            s = chunk_inputs(chunks, [whole - 3, half], 8, 2, D, q_dt, cache, 180 + bq, NB=NB, bq=bq, topk=topk, per_head=per_head)
            if bq:
                pick = s["topk"] if per_head else s["topk"][:1].clone()
                pick[:, 0, 1:3] = torch.tensor([NB - 1, NB - 2], dtype=I32)
                pick[:, -1, 1:4] = torch.tensor([NB, NB - 1, 31], dtype=I32)
                s["topk"] = pick if per_head else pick.expand(2, -1, -1)
            run_chunk(spd, s, what="NB %d bq %d" % (NB, bq))


@pytest.mark.parametrize("NB", [129, 1024])
def test_whole_chunks_over_long_page_tables(spd, NB):
    """Chunks of several pairs over every key of a long table, among short
    ones."""
    for cache in (E4M3, BF16):
        s = chunk_inputs([35, 5, 17], [NB * BS - 35, 300, 9000], 8, 1, 128, BF16, cache, 190, NB=NB)
        run_chunk(spd, s, what="NB %d" % NB)


@pytest.mark.parametrize("NB", [25, 1024])
def test_assign_long_page_tables(spd, NB):
    g = torch.Generator().manual_seed(NB)
    B, cap = 70, NB * BS
    prefix = torch.randint(0, cap + 300, (B,), generator=g).tolist()
    new = torch.randint(0, 3000, (B,), generator=g).tolist()
    prefix[:5], new[:5] = [cap - 1, cap, cap - 128, 0, cap - 127], [1, 7, 128, min(cap, 100000), 129]
    rows = torch.randperm(B + 3, generator=g)[:B].to(I32)
    table = torch.randperm((B + 3) * NB, generator=g).to(I32).view(B + 3, NB)
    grown = sum(-(-min(p + n, cap) // BS) - -(-min(p, cap) // BS) for n, p in zip(new, prefix))
    free = (torch.randperm(grown + 9, generator=g) + (B + 3) * NB).to(I32)
    T = sum(new) + 11
    for count in (grown + 9, grown - 20):
        args = (i32(new), i32(prefix), rows.to(DEV), free.to(DEV), i32([count]), (B + 3) * NB + grown + 9, 64, table.to(DEV), T)
        check_assign(run_assign(spd, *args), *args, "NB %d" % NB)


# ------------------------------------------------------------- large logits


@pytest.mark.parametrize("kind", KINDS)
def test_logits_of_tens_of_millions(spd, kind):
    """Two keys of weight in the halves of a page, the second's logit a little
    larger, both so large that their 32-bit spacing is 1 to 4: their weights
    are anything, and their values the same, so the output is that value."""
    D, q_dt, cache = kind_of(kind)
    s = chunk_inputs([96], [200], 16, 2, D, q_dt, cache, 200)
    s["q"].zero_()
    row = torch.arange(96 * 16).view(96, 16)
    s["q"][..., 0] = (20000.0 + 26.0 * row).to(q_dt)  # logits of 9 to 26.9 millions
    s["q"][..., 1] = (3.0 + row % 7).to(q_dt)
    page = s["owned"][0].tolist()
    code = (lambda x: torch.tensor(x).to(E4M3).view(torch.uint8).item()) if cache == E4M3 else (lambda x: x)
    kc = s["kc"].view(torch.uint8) if cache == E4M3 else s["kc"]
    for p in page:
        kc[p * BS:(p + 1) * BS] = 0
    kc[page[0] * BS + 5, :, 0], kc[page[0] * BS + 90, :, 0] = code(448.0), code(448.0)
    kc[page[0] * BS + 90, :, 1] = code(1.0)
    vc = s["vc"].view(torch.uint8) if cache == E4M3 else s["vc"]
    vc[page[0] * BS + 90] = vc[page[0] * BS + 5]
    s["ks"], s["sm"] = 1.0, 1.0
    run_chunk(spd, s, what="large logits")


# ------------------------------------------------------ a step as one graph


@pytest.mark.parametrize("cache", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_a_captured_step_goes_on_by_itself(spd, cache):
    """Slots, stores, selection and attention captured in one graph that also
    carries the lengths and the free count over: each replay is the next step
    of the loop, with new lengths, and leaves what the same calls one by one
    leave."""
    B, Hq, Hkv, D, NB, bq, K, T = 4, 16, 2, 128, 16, 16, 4, 700
    pool, rows_cap = 80, 700 // 16 + 4
    ks = vs = 0.02 if cache == E4M3 else 1.0
    g = torch.Generator().manual_seed(11)
    angle = torch.rand((NB * BS, D // 2), generator=g, dtype=torch.float64) * 6.3
    fixed = dict(rows=i32([2, 0, 4, 1]), free=torch.randperm(pool, generator=g).to(I32).to(DEV),
                 w=(1 + 0.1 * torch.randn(D, generator=g)).to(BF16).to(DEV),
                 cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV))

    def state():
        kv = [torch.full((pool * BS, Hkv, D), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3) if cache == E4M3 else
              torch.full((pool * BS, Hkv, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2)]
        s = dict(new=i32([0] * B), prefix=i32([0] * B), count=i32([pool]), x=torch.zeros((T, Hq + 2 * Hkv + 3, D), dtype=BF16, device=DEV),
                 table=torch.full((5, NB), -1, dtype=I32, device=DEV), kc=kv[0], vc=kv[1],
                 kic=torch.full((pool * BS, 1, D), float("nan"), dtype=BF16, device=DEV),
                 q=nan_like((T, Hq, D), BF16, DEV), qi=nan_like((T, 2, D), BF16, DEV), o=nan_like((T, Hq, D), BF16, DEV),
                 dense=nan_like((T, Hq, D), BF16, DEV), topk=nan_like((2, rows_cap, K), I32, DEV))
        for n, size in (("cu", B + 1), ("cub", B + 1), ("sl", B), ("req", T), ("lens", T), ("slots", T), ("left", 1)):
            s[n] = nan_like((size,), I32, DEV)
        s["was"] = i32([0] * B)
        s["pws"] = torch.empty(spd.prefill_workspace_bytes(T, 2, NB), dtype=torch.uint8, device=DEV)
        s["ws"] = torch.empty(spd.prefill_attention_workspace_bytes(T, Hq, Hkv, D, B, NB, rows_cap), dtype=torch.uint8, device=DEV)
        return s

    def step(s):
        f, x = fixed, s["x"]
        s["was"].copy_(s["prefix"])
        spd.paged_assign_slots(s["new"], s["prefix"], f["rows"], f["free"], s["count"], pool, BS, bq, s["table"], s["cu"], s["cub"],
                               s["sl"], s["req"], s["lens"], s["slots"], s["left"])
        spd.paged_norm_rope_store(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv], f["w"], f["w"], f["cos_sin"], s["lens"],
                                  s["slots"], s["q"], s["kc"], s["vc"], 1e-6, False, BS, ks, vs)
        spd.paged_norm_rope_store(x[:, -3:-1], x[:, -1:], None, f["w"], f["w"], f["cos_sin"], s["lens"], s["slots"], s["qi"],
                                  s["kic"], None, 1e-6, False, BS, 1.0, 1.0)
        spd.msa_prefill_block_score(s["qi"], s["kic"], s["table"], f["rows"], s["cu"], s["sl"], s["prefix"], bq, BS, 1, 1, D ** -0.5,
                                    s["cub"], s["topk"], s["pws"])
        head = (s["q"], s["kc"], s["vc"], s["table"], f["rows"], s["cu"], s["sl"], s["prefix"])
        spd.paged_sparse_prefill_attention(*head, s["topk"], bq, s["cub"], s["o"], D ** -0.5, BS, ks, vs, s["ws"])
        spd.paged_prefill_attention(*head, s["dense"], D ** -0.5, BS, ks, vs, s["ws"])
        s["prefix"].copy_(s["sl"])
        s["count"].copy_(s["left"])

    warm = state()
    step(warm)  # a step of no tokens; before any capture
    a, b = state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    torch.cuda.synchronize()
    for n, new in enumerate(([300, 1, 0, 17], [1, 200, 0, 300], [0, 0, 0, 0], [1, 1, 1, 1], [128, 400, 127, 60])):
        x = torch.randn(tuple(a["x"].shape), generator=g).to(BF16).to(DEV)
        for s in (a, b):
            s["new"].copy_(i32(new))
            s["x"].copy_(x)
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for name in a:
            if name not in ("ws", "pws"):
                assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), "step %d: %s" % (n, name)
        for out, topk in ((a["o"], a["topk"]), (a["dense"], None)):
            ref, A = R.attention(a["q"], a["kc"], a["vc"], a["table"], fixed["rows"], a["cu"], a["sl"], a["was"], D ** -0.5, ks, vs,
                                 topk, bq, a["cub"])
            R.check_attention(out, ref, A, "step %d" % n)
        assert spd.workspace_status(a["ws"]) == 0
