"""The block-scaled E4M3 caches on the GPU: their store and the attention that
reads them, against the 64-bit definitions and tolerances of block_scaled_ref.py.

Outputs are poisoned before each call, inputs hashed before and after; slots and
scales that no request owns hold NaN, so that a value read from one shows.
"""
import random

import numpy as np
import pytest
import torch

import block_scaled_ref as B
import serve_ref as R
from parity import digest, nan_like

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BS = 128
I32 = torch.int32
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def spd():
    import sparse_paged_decode_gb300 as m

    return m


@pytest.fixture(params=[0, 1], ids=["default", "general"])
def store_kernel(spd, request):
    old = spd.set_kernel_policy(6, request.param)
    yield request.param
    spd.set_kernel_policy(6, old)


def i32(values):
    return torch.tensor(values, dtype=I32, device=DEV)


def codes(shape, g, cache_nan=False):
    x = torch.randn(shape, generator=g) * 60.0
    return x.clamp(-448, 448).to(E4M3)


# -------------------------------------------------------------------- store


def store_inputs(parts, Hq, Hkv, D, Rd, dt, seed, weights=BF16, pad=0, spread=6, pads_at=None):
    """`parts`: (prefix, new tokens) of each request, on shuffled pages.  Heads
    differ in magnitude by powers of two, so some pages grow and some do not."""
    g = torch.Generator().manual_seed(seed)
    owned = [-(-(p + n) // BS) for p, n in parts]
    pool = sum(owned) + 3
    perm = torch.randperm(pool, generator=g).tolist()
    lens, slots, at = [], [], 0
    for (p, n), own in zip(parts, owned):
        pages = perm[at:at + own]
        at += own
        lens += [p + i + 1 for i in range(n)]
        slots += [pages[(p + i) // BS] * BS + (p + i) % BS for i in range(n)]
        if pads_at == "between":  # a padding row behind each request
            lens.append(0)
            slots.append(-1)
    lens += [0] * pad
    slots += [-1] * pad
    T, M = len(lens), max([p + n for p, n in parts] + [1]) + 1
    mags = torch.exp2(torch.randint(-spread, spread + 1, (1, Hq + 2 * Hkv, 1), generator=g).float())
    fused = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * mags).to(dt).to(DEV)
    angle = torch.rand((M, Rd // 2), generator=g, dtype=torch.float64) * 6.3
    s = dict(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:],
             wq=None if weights is None else (1 + 0.2 * torch.randn(D, generator=g)).to(weights).to(DEV),
             wk=None if weights is None else (1 + 0.2 * torch.randn(D, generator=g)).to(weights).to(DEV),
             cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV), lens=i32(lens), slots=i32(slots))
    for name in ("k", "v"):
        s[name + "c"] = codes((pool * BS, Hkv, D), g).to(DEV)
        s[name + "s"] = torch.exp2(torch.randint(-12, 3, (pool, Hkv), generator=g).float()).to(DEV)
    return s


CACHES = ("kc", "vc", "ks", "vs")


def run_store(spd, s, out_dt=None, eps=1e-6, interleaved=False, out=None):
    if out is None:
        out = nan_like(tuple(s["q"].shape), out_dt or s["q"].dtype, DEV)
    ins = [s[n] for n in ("q", "k", "v", "wq", "wk", "cos_sin", "lens", "slots")]
    before = digest(*[x for x in ins if x is not None])
    spd.paged_norm_rope_store_block_scaled(*ins, out, *[s[n] for n in CACHES], eps, interleaved, BS)
    torch.cuda.synchronize()
    assert digest(*[x for x in ins if x is not None]) == before, "inputs mutated"
    return out


def check_store(spd, s, what, out_dt=None, eps=1e-6, interleaved=False, again=True, out=None):
    before = {n: B.kept(s[n]) for n in CACHES}
    got = run_store(spd, s, out_dt, eps, interleaved, out)
    after = {n: B.kept(s[n]) for n in CACHES}
    B.check_store(s, before, after, got, eps, interleaved, what)
    if again:  # the same call once more leaves the caches as they are
        run_store(spd, s, out_dt, eps, interleaved, out)
        for n in CACHES:
            assert np.array_equal(B.kept(s[n]), after[n], equal_nan=True), "%s: a second call changed %s" % (what, n)


STORE = [
    dict(parts=[(0, 1)]),
    dict(parts=[(127, 1), (128, 1), (129, 1), (1, 1)], Hq=4, Hkv=4),
    dict(parts=[(0, 128)], Hq=1, Hkv=1),
    dict(parts=[(0, 129), (1, 127), (100, 300)], Hq=16, Hkv=2, pad=3),
    dict(parts=[(5, 1), (200, 4), (127, 8), (250, 16), (0, 16)], Hq=64, Hkv=8, pads_at="between"),
    dict(parts=[(77, 300), (13, 1), (640, 511)], Hq=6, Hkv=3, D=64, Rd=64),
    dict(parts=[(77, 130), (13, 1), (0, 0), (3, 5)], Hq=8, Hkv=8, D=256, Rd=128),
    dict(parts=[(30, 100), (0, 7)], Hq=24, Hkv=3, D=128, Rd=64),
    dict(parts=[(30, 100), (0, 7)], Hq=5, Hkv=5, D=40, Rd=12),
    dict(parts=[(30, 33)], Hq=3, Hkv=1, D=1 + 1, Rd=2),
    dict(parts=[(p, 1) for p in range(0, 640, 7)], Hq=8, Hkv=1),
    dict(parts=[(p, 2 + p % 3) for p in range(0, 1270, 9)], Hq=8, Hkv=2, pad=40),
    dict(parts=[], pad=4),
]


@pytest.mark.parametrize("kind", [(BF16, False, BF16), (F16, True, F32), (F32, False, None)], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("i", range(len(STORE)))
def test_store(spd, store_kernel, i, kind):
    dt, inter, weights = kind
    c = dict(STORE[i])
    D = c.pop("D", 128)
    s = store_inputs(c.pop("parts"), c.pop("Hq", 8), c.pop("Hkv", 2), D, c.pop("Rd", D), dt, 100 + i, weights=weights, **c)
    check_store(spd, s, "case %d" % i, interleaved=inter)


@pytest.mark.parametrize("shape", [(8, 2, 128), (6, 3, 64), (2, 2, 256), (3, 1, 48)])
def test_store_not_finite_and_out_of_range(spd, store_kernel, shape):
    Hq, Hkv, D = shape
    s = store_inputs([(60, 100), (0, 3), (126, 9), (40, 2)], Hq, Hkv, D, D, BF16, 7, weights=None)
    s["v"][3, 0, 5], s["v"][4, 0, 1], s["v"][90, Hkv - 1, 2] = float("nan"), float("inf"), float("-inf")
    s["v"][100:103] = 0.0                       # a page that is begun with zeros
    s["v"][103:112, 0] = torch.finfo(BF16).max  # above 448 * 2^64: saturates
    s["v"][112:, 0] = 2.0 ** -100               # below the smallest scale
    s["k"][103:112] = 0.0
    s["vs"][int(s["slots"][103]) // BS, 0] = float("nan")  # no scale that could have scaled anything
    s["vs"][int(s["slots"][112]) // BS] = 0.0
    s["ks"][int(s["slots"][112]) // BS] = float("inf")
    check_store(spd, s, "not finite", again=False)


@pytest.mark.parametrize("old", [3e-39, 0.7, 1.1, 5.0, 3e38])
def test_store_keeps_or_replaces_any_scale(spd, store_kernel, old):
    """Scales of another maker: kept where they are large enough, else replaced by a power of two."""
    s = store_inputs([(60, 30), (5, 200)], 4, 2, 128, 128, BF16, 8)
    s["ks"].fill_(old)
    s["vs"].fill_(old)
    check_store(spd, s, "old scale %g" % old)


def test_store_borders_of_the_scales(spd, store_kernel):
    """Largest values at and next to 448 * 2^e, for V exactly known."""
    s = store_inputs([(9, 1) for _ in range(12)], 2, 2, 128, 128, F32, 9, weights=None)
    s["vs"].fill_(2.0 ** -40)
    s["v"].zero_()
    for t in range(12):
        x = torch.tensor(448.0 * 2.0 ** (t - 6))
        s["v"][t, 0, 17] = x
        s["v"][t, 1, 64] = -torch.nextafter(x, torch.tensor(1e30))
    check_store(spd, s, "borders")
    page = s["slots"].long() // BS
    want = torch.exp2(torch.arange(12, device=DEV).float() - 6)
    assert torch.equal(s["vs"][page, 0], want) and torch.equal(s["vs"][page, 1], 2 * want)


@pytest.mark.parametrize("kind", ["padded", "dims", "interleaved", "scales", "inputs"])
def test_store_strides(spd, store_kernel, kind):
    s = store_inputs([(60, 100), (0, 3), (126, 9)], 8, 2, 128, 128, BF16, 11)
    P = s["ks"].shape[0]
    out = None
    if kind == "padded":
        for n in ("kc", "vc"):
            big = torch.zeros((P * BS, 3, 160), dtype=torch.uint8, device=DEV).view(E4M3)
            big[:, :2, :128].view(torch.uint8).copy_(s[n].view(torch.uint8))
            s[n] = big[:, :2, :128]
    elif kind == "dims":
        for n in ("kc", "vc"):
            big = torch.zeros((P * BS, 2, 256), dtype=torch.uint8, device=DEV)
            big[:, :, ::2] = s[n].view(torch.uint8)
            s[n] = big.view(E4M3)[:, :, ::2]
        out = nan_like((s["q"].shape[0], 128, 8), BF16, DEV).transpose(1, 2)
    elif kind == "interleaved":
        both = torch.stack((s["kc"].view(torch.uint8), s["vc"].view(torch.uint8)), 1).contiguous().view(E4M3)
        s["kc"], s["vc"] = both[:, 0], both[:, 1]
    elif kind == "scales":
        for n in ("ks", "vs"):
            s[n] = s[n].t().contiguous().t()
    else:
        s["k"] = s["k"].flip(0).flip(0).transpose(0, 1).contiguous().transpose(0, 1)
        s["v"] = s["v"][:, :1].expand(-1, 2, -1)  # a broadcast input
        s["lens"] = torch.stack((s["lens"], s["lens"]), 1)[:, 0]
    check_store(spd, s, kind, out=out)


def test_store_slots_outside_the_pool_and_positions_outside_the_table(spd, store_kernel):
    s = store_inputs([(60, 100), (0, 30), (126, 9)], 8, 2, 128, 128, BF16, 12)
    P, M = s["ks"].shape[0], s["cos_sin"].shape[0]
    s["slots"][20], s["slots"][110], s["lens"][105], s["lens"][2] = P * BS, -7, M + 1, -5
    # a row that is left out ends a run: what follows it on the same page must be dropped too
    s["slots"][3:68], s["slots"][21:68] = -1, -1
    s["slots"][106:130] = -1
    check_store(spd, s, "outside")


def test_store_many_rows(spd, store_kernel):
    r = random.Random(3)
    parts = [(r.randint(0, 400), r.choice((1, 1, 2, 4, 16, 130, 257))) for _ in range(150)]
    s = store_inputs(parts, 4, 2, 64, 64, BF16, 13, pads_at="between", pad=100)
    check_store(spd, s, "many rows")


# ---------------------------------------------------------------- attention


def attention_inputs(lengths, new, Hq, Hkv, D, dt, seed, NB=None, K=0, bq=1, spread=4, wild=0, pad=0, general=False):
    """Requests of `lengths` keys whose last `new` tokens are the queries.  Slots and
    pages that no request owns hold NaN codes and NaN scales."""
    g = torch.Generator().manual_seed(seed)
    n = len(lengths)
    owned = [-(-L // BS) for L in lengths]
    NB = NB or max(owned + [1])
    pool = sum(owned) + 4
    perm = torch.randperm(pool, generator=g)
    table = torch.full((n + 2, NB), -1, dtype=I32)
    rows = torch.randperm(n + 2, generator=g)[:n].to(I32)
    free, at = perm[sum(owned):], 0
    out = {}
    for name in ("k", "v"):
        c = codes((pool * BS, Hkv, D), g)
        if name == "k":  # logits of a few units
            c = (c.float() / 30).to(E4M3)
        scale = torch.exp2(torch.randint(-spread, spread + 1, (pool, Hkv), generator=g).float()) if name == "v" else torch.exp2(
            torch.randint(-1, 2, (pool, Hkv), generator=g).float())
        if general:
            scale = scale * (0.6 + torch.rand((pool, Hkv), generator=g))
        if wild and name == "v":
            scale = torch.exp2(torch.randint(-wild, wild + 1, (pool, Hkv), generator=g).float())
        out[name + "c"], out[name + "s"] = c, scale
    for b, (L, own) in enumerate(zip(lengths, owned)):
        pages = perm[at:at + own]
        at += own
        table[rows[b], :own] = pages.to(I32)
        table[rows[b], own:] = free[0].to(I32)
        if L % BS:
            for name in ("kc", "vc"):
                out[name].view(torch.uint8)[pages[-1] * BS + L % BS:(pages[-1] + 1) * BS] = 0x7F
    for page in free.tolist():
        for name in ("k", "v"):
            out[name + "c"].view(torch.uint8)[page * BS:(page + 1) * BS] = 0x7F
            out[name + "s"][page] = float("nan")
    cu = [0]
    for c in new:
        cu.append(cu[-1] + c)
    T = cu[-1] + pad
    out.update(table=table, rows=rows, cu=torch.tensor(cu, dtype=I32), seq_lens=torch.tensor(lengths, dtype=I32),
               prefix=torch.tensor([L - c for L, c in zip(lengths, new)], dtype=I32),
               q=torch.randn((T, Hq, D), generator=g).to(dt))
    out["lens"] = torch.tensor([L - c + i + 1 for L, c in zip(lengths, new) for i in range(c)] + [0] * pad, dtype=I32)
    out["req"] = torch.tensor([int(rows[b]) for b, c in enumerate(new) for _ in range(c)] + [-1] * pad, dtype=I32)
    out = {k: v.to(DEV) for k, v in out.items()}
    out.update(sm=D ** -0.5, Hkv=Hkv, bq=bq, topk=None, cub=None, NB=NB)
    if K:
        cub = [0]
        for c in new:
            cub.append(cub[-1] + -(-c // bq))
        n_rows = cub[-1] + (pad if bq == 1 else 0)
        tk = torch.randint(-1, NB + 1, (Hkv, n_rows, K), generator=g).to(I32)
        tk[:, ::3, 0] = 0
        out["topk"], out["cub"] = tk.to(DEV), i32(cub)
    return out


def run_decode(spd, s, policy=None, out=None, ws=None):
    T, Hq, D = s["q"].shape
    out = nan_like((T, Hq, D), BF16, DEV) if out is None else out
    if ws is None:
        ws = torch.randint(0, 256, (spd.decode_workspace_bytes(T, Hq, s["Hkv"], D, s["NB"]),), dtype=torch.uint8, device=DEV)
        ws[:256] = 0  # the status word, which only the tensor-core kernels write
    ins = [s[n] for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "req")] + ([s["topk"]] if s["topk"] is not None else [])
    before = digest(*ins)
    old = spd.set_kernel_policy(3, policy) if policy is not None else None
    try:
        f = spd.paged_decode_attention_block_scaled if s["topk"] is None else spd.paged_sparse_decode_attention_block_scaled
        f(*ins, out, s["sm"], BS, ws)
    finally:
        if policy is not None:
            spd.set_kernel_policy(3, old)
    torch.cuda.synchronize()
    assert digest(*ins) == before, "inputs mutated"
    if ws.numel() and policy != 1:
        assert spd.workspace_status(ws) & 1 == 0 or T == 0, "a wait gave up"
    return out


def run_prefill(spd, s, policy=None, out=None, ws=None):
    T, Hq, D = s["q"].shape
    out = nan_like((T, Hq, D), BF16, DEV) if out is None else out
    n_rows = s["topk"].shape[1] if s["topk"] is not None else 0
    if ws is None:
        size = spd.prefill_attention_workspace_bytes(T, Hq, s["Hkv"], D, s["rows"].numel(), s["NB"], n_rows)
        ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV)
    ins = [s[n] for n in ("q", "kc", "vc", "ks", "vs", "table", "rows", "cu", "seq_lens", "prefix")]
    more = [] if s["topk"] is None else [s["topk"], s["bq"], s["cub"]]
    before = digest(*ins, *[x for x in more if torch.is_tensor(x)])
    old = spd.set_kernel_policy(5, policy) if policy is not None else None
    try:
        f = spd.paged_prefill_attention_block_scaled if s["topk"] is None else spd.paged_sparse_prefill_attention_block_scaled
        f(*ins, *more, out, s["sm"], BS, ws)
    finally:
        if policy is not None:
            spd.set_kernel_policy(5, old)
    torch.cuda.synchronize()
    assert digest(*ins, *[x for x in more if torch.is_tensor(x)]) == before, "inputs mutated"
    if T:
        assert spd.workspace_status(ws) & 1 == 0, "a wait gave up"
    return out


def check_decode(spd, s, policies, what):
    ref = B.decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["req"], s["sm"], s["topk"])
    for pol in policies:
        B.check_attention(run_decode(spd, s, pol), *ref, "%s, policy %s" % (what, pol))


def check_prefill(spd, s, policies, what):
    ref = B.attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["rows"], s["cu"], s["seq_lens"], s["prefix"],
                      s["sm"], s["topk"], s["bq"], s["cub"])
    for pol in policies:
        B.check_attention(run_prefill(spd, s, pol), *ref, "%s, policy %s" % (what, pol))


DECODE = [
    dict(lengths=[1], new=[1], Hq=8, Hkv=1),
    dict(lengths=[127, 128, 129, 1], new=[1, 1, 1, 1], Hq=64, Hkv=8),
    dict(lengths=[300, 517, 1100, 40], new=[4, 16, 1, 8], Hq=16, Hkv=2, pad=3),
    dict(lengths=[900, 77], new=[3, 2], Hq=4, Hkv=4),
    dict(lengths=[900, 77], new=[16, 1], Hq=32, Hkv=2),
    dict(lengths=[2500] * 3, new=[16, 16, 16], Hq=8, Hkv=1),
    dict(lengths=[6000], new=[1], Hq=8, Hkv=1),
    dict(lengths=[300, 200], new=[4, 1], Hq=6, Hkv=2),
    dict(lengths=[300, 200], new=[4, 1], Hq=8, Hkv=2, D=64),
    dict(lengths=[300, 200], new=[4, 1], Hq=5, Hkv=5, D=48),
    dict(lengths=[400, 260], new=[2, 2], Hq=8, Hkv=2, NB=300),
]


@pytest.mark.parametrize("dt", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [0, 3])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(spd, i, K, dt):
    c = dict(DECODE[i])
    s = attention_inputs(c.pop("lengths"), c.pop("new"), c.pop("Hq"), c.pop("Hkv"), c.pop("D", 128), dt, 200 + i, K=K,
                         general=i % 2 == 1, **c)
    check_decode(spd, s, (None, 1, 2, 3, 4), "case %d" % i)


@pytest.mark.parametrize("pol", [None, 1, 2, 3, 4])
@pytest.mark.parametrize("K", [0, 5])
def test_decode_scales_far_apart(spd, K, pol):
    s = attention_inputs([1500, 260, 640], [4, 1, 8], 16, 2, 128, BF16, 31, K=K, wild=24)
    check_decode(spd, s, (pol,), "far apart")


@pytest.mark.parametrize("pol", [None, 1, 2, 3, 4])
def test_decode_scales_outside_the_range(spd, pol):
    """0, negative and NaN count as 2^-64, what is above 2^64 as that."""
    s = attention_inputs([1500, 260, 640], [4, 1, 8], 16, 2, 128, BF16, 32)
    t = s["table"][s["rows"].long()].long()
    for j, bad in enumerate((0.0, -3.0, float("nan"), 1e-30)):
        s["ks"][t[0, j]] = bad
        s["vs"][t[0, j + 4]] = bad
    s["vs"][t[1]] = 2.0 ** 70
    s["vs"][t[2]] = 1e-38
    check_decode(spd, s, (pol,), "outside")


def test_decode_bad_metadata(spd):
    """Rows outside the table, pages outside the pool, lengths past the table."""
    for pol in (None, 1, 2, 3, 4):
        s = attention_inputs([700, 300, 900], [2, 2, 2], 16, 2, 128, BF16, 33)
        s["req"][0], s["req"][1] = -1, 99
        s["table"][s["rows"][1].long(), 1] = -5
        s["table"][s["rows"][2].long(), 0] = s["ks"].shape[0]
        s["lens"][4:] = 5000
        s["kc"].view(torch.uint8)[s["kc"].view(torch.uint8) == 0x7F] = 0
        s["vc"].view(torch.uint8)[s["vc"].view(torch.uint8) == 0x7F] = 0
        s["ks"].nan_to_num_(nan=1.0)
        s["vs"].nan_to_num_(nan=1.0)
        check_decode(spd, s, (pol,), "metadata")


PREFILL = [
    dict(lengths=[1], new=[1], Hq=8, Hkv=1),
    dict(lengths=[127, 128, 129, 513], new=[127, 1, 129, 100], Hq=16, Hkv=2),
    dict(lengths=[900, 300, 1300], new=[16, 0, 5], Hq=64, Hkv=8, pad=2),
    dict(lengths=[3000], new=[3], Hq=8, Hkv=1),
    dict(lengths=[2000, 400], new=[200, 333], Hq=8, Hkv=4),
    dict(lengths=[2000, 400], new=[70, 33], Hq=8, Hkv=2, D=64),
    dict(lengths=[700, 400], new=[7, 33], Hq=6, Hkv=2),
    dict(lengths=[700, 400], new=[7, 33], Hq=4, Hkv=4, D=96),
    dict(lengths=[700, 400], new=[7, 33], Hq=16, Hkv=1, NB=600),
]


@pytest.mark.parametrize("dt", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("bq", [0, 1, 16, 100])
@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill(spd, i, bq, dt):
    c = dict(PREFILL[i])
    s = attention_inputs(c.pop("lengths"), c.pop("new"), c.pop("Hq"), c.pop("Hkv"), c.pop("D", 128), dt, 300 + i,
                         K=3 if bq else 0, bq=max(bq, 1), general=i % 2 == 1, **c)
    check_prefill(spd, s, (None, 1), "case %d" % i)


@pytest.mark.parametrize("pol", [None, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bq", [0, 16])
def test_prefill_scales_far_apart(spd, bq, D, pol):
    s = attention_inputs([1500, 260, 640], [40, 10, 300], 16, 2, D, BF16, 34, K=5 if bq else 0, bq=max(bq, 1), wild=24)
    check_prefill(spd, s, (pol,), "far apart")


@pytest.mark.parametrize("pol", [None, 1])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_prefill_scales_outside_the_range(spd, dt, pol):
    s = attention_inputs([1500, 260, 640], [4, 1, 8], 16, 2, 128, dt, 35)
    t = s["table"][s["rows"].long()].long()
    for j, bad in enumerate((0.0, -3.0, float("nan"), 1e-30)):
        s["ks"][t[0, j]] = bad
        s["vs"][t[0, j + 4]] = bad
    s["vs"][t[1]] = 2.0 ** 70
    s["vs"][t[2]] = 1e-38
    check_prefill(spd, s, (pol,), "outside")


@pytest.mark.parametrize("pol", [None, 1])
def test_rows_of_one_small_block_and_heavy_logits(spd, pol):
    """A row whose weight lies on a block of a tiny value scale, beside a block of a large one with logits far below."""
    s = attention_inputs([256], [1], 8, 1, 128, BF16, 36)
    t = s["table"][s["rows"][0].long()].long()
    s["q"].fill_(1.0)
    for j, code in enumerate((4.0, -4.0)):  # logits +-45
        s["kc"][t[j] * BS:(t[j] + 1) * BS] = torch.full((BS, 1, 128), code, device=DEV).to(E4M3)
    s["ks"].fill_(1.0)
    s["vs"][t[0]], s["vs"][t[1]] = 2.0 ** -40, 2.0 ** 30
    check_prefill(spd, s, (pol,), "prefill")
    check_decode(spd, s, (None, 1, 2, 3, 4), "decode")


@pytest.mark.parametrize("K", [0, 3])
@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_strided_operands(spd, which, K):
    s = attention_inputs([700, 300], [4, 2], 16, 2, 128, BF16, 37, K=K)
    s["ks"] = s["ks"].t().contiguous().t()
    s["vs"] = torch.stack((s["vs"], s["vs"]), 2)[:, :, 1]
    both = torch.stack((s["kc"].view(torch.uint8), s["vc"].view(torch.uint8)), 1).contiguous().view(E4M3)
    s["kc"], s["vc"] = both[:, 0], both[:, 1]
    s["q"] = s["q"].transpose(0, 1).contiguous().transpose(0, 1)
    (check_decode if which == "decode" else check_prefill)(spd, s, (None, 1), "strided")
    for n in ("kc", "vc"):  # slots 16 bytes apart from their own width: the general kernels
        big = torch.zeros((s[n].shape[0], 2, 136), dtype=torch.uint8, device=DEV)
        big[:, :, :128] = s[n].view(torch.uint8)
        s[n] = big.view(E4M3)[:, :, :128]
    (check_decode if which == "decode" else check_prefill)(spd, s, (None,), "odd rows")


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_empty_batches(spd, which):
    s = attention_inputs([300], [0], 8, 1, 128, BF16, 38)
    (run_decode if which == "decode" else run_prefill)(spd, s)
    s = attention_inputs([300, 1], [0, 0], 8, 1, 128, BF16, 38, pad=3)
    assert not (run_decode if which == "decode" else run_prefill)(spd, s).float().any()


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_scales_of_one_agree_with_the_static_call(spd, which, dt):
    s = attention_inputs([1700, 300, 129], [4, 2, 16], 64, 8, 128, dt, 39)
    s["ks"].fill_(0.5)
    s["vs"].fill_(0.25)
    T, Hq, D = s["q"].shape
    other = nan_like((T, Hq, D), BF16, DEV)
    if which == "decode":
        got = run_decode(spd, s)
        ws = torch.empty(spd.decode_workspace_bytes(T, Hq, 8, D, s["NB"]), dtype=torch.uint8, device=DEV)
        spd.paged_decode_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["req"], other, s["sm"], BS, 0.5, 0.25, ws)
    else:
        got = run_prefill(spd, s)
        ws = torch.empty(spd.prefill_attention_workspace_bytes(T, Hq, 8, D, 3, s["NB"]), dtype=torch.uint8, device=DEV)
        spd.paged_prefill_attention(s["q"], s["kc"], s["vc"], s["table"], s["rows"], s["cu"], s["seq_lens"], s["prefix"], other,
                                    s["sm"], BS, 0.5, 0.25, ws)
    # each is within its bound of the exact output
    ref = B.decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["req"], s["sm"])
    B.check_attention(got, *ref, "block-scaled")
    B.check_attention(other, *ref, "static")


# ------------------------------------------------------------ runs of calls


def test_far_pages_of_a_large_cache(spd):
    """Offsets past 2^31 bytes: pages at the end of a cache of 20000 pages of 1 KiB slots."""
    P, Hkv, D = 20000, 8, 128
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.zeros((P * BS, Hkv, D), dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ks, vs = (torch.full((P, Hkv), float("nan"), device=DEV) for _ in range(2))
    pages = [19998, 3, 19999]
    L = 300
    T = L
    lens = i32(list(range(1, L + 1)))
    slots = i32([pages[i // BS] * BS + i % BS for i in range(L)])
    fused = torch.randn((T, 64 + 2 * Hkv, D), generator=g).to(BF16).to(DEV)
    angle = torch.rand((L, D // 2), generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV)
    out = nan_like((T, 64, D), BF16, DEV)
    spd.paged_norm_rope_store_block_scaled(fused[:, :64], fused[:, 64:72], fused[:, 72:], None, None, cs, lens, slots, out, kc, vc,
                                           ks, vs, 1e-6, False, BS)
    torch.cuda.synchronize()
    k, mag = R.head_rows(fused[:, 64:72], None, cs, R.ints(lens), 1e-6, False)
    got = B.kept(kc[slots.long()].float()) * B.kept(ks[slots.long() // BS])[:, :, None]
    top = np.abs(k).max()
    assert np.abs(got - k).max() <= 2.0 ** -4 * top + 1e-6
    assert not kc.view(torch.uint8)[:3 * BS].any() and bool(torch.isnan(ks[:3]).all())
    small = dict(q=out[-5:].contiguous(), Hkv=Hkv, NB=3, sm=D ** -0.5, topk=None, cub=None, bq=1, table=i32([pages]),
                 rows=i32([0]), cu=i32([0, 5]), seq_lens=i32([L]), prefix=i32([L - 5]), lens=lens[-5:].contiguous(), req=i32([0] * 5))
    near = torch.cat([torch.arange(p * BS, (p + 1) * BS) for p in pages]).to(DEV)
    ref_in = (small["q"], kc[near], vc[near], ks[pages], vs[pages], i32([[0, 1, 2]]))
    ref = B.decode(*ref_in, small["lens"], small["req"], small["sm"])
    small.update(kc=kc, vc=vc, ks=ks, vs=vs)
    T5, Hq = 5, 64
    ws = torch.empty(max(spd.decode_workspace_bytes(T5, Hq, Hkv, D, 3), spd.prefill_attention_workspace_bytes(T5, Hq, Hkv, D, 1, 3)),
                     dtype=torch.uint8, device=DEV)
    o1, o2 = nan_like((5, 64, D), BF16, DEV), nan_like((5, 64, D), BF16, DEV)
    spd.paged_decode_attention_block_scaled(small["q"], kc, vc, ks, vs, small["table"], small["lens"], small["req"], o1, small["sm"], BS, ws)
    torch.cuda.synchronize()
    B.check_attention(o1, *ref, "decode")
    spd.paged_prefill_attention_block_scaled(small["q"], kc, vc, ks, vs, small["table"], small["rows"], small["cu"], small["seq_lens"],
                                             small["prefix"], o2, small["sm"], BS, ws)
    torch.cuda.synchronize()
    B.check_attention(o2, *ref, "prefill")


def test_a_serving_loop(spd):
    """assign -> store -> attention for a prefill step and several decode steps, each captured once as a graph or called."""
    Hq, Hkv, D, NB, F, n = 16, 2, 128, 8, 64, 3
    g = torch.Generator().manual_seed(11)
    kc, vc = (torch.full((F * BS, Hkv, D), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ks, vs = (torch.full((F, Hkv), float("nan"), device=DEV) for _ in range(2))
    table = torch.full((5, NB), -1, dtype=I32, device=DEV)
    rows, prefix = i32([4, 0, 2]), i32([0, 0, 0])
    free, count = torch.randperm(F, generator=g).to(I32).to(DEV), i32([F])
    M = NB * BS
    angle = torch.rand((M, D // 2), generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(BF16).to(DEV)
    lengths = [0, 0, 0]
    for step, new in enumerate(([200, 1, 127], [1, 4, 1], [4, 130, 2], [1, 1, 16], [0, 1, 1])):
        T = sum(new) + 3
        one = dict(dtype=I32, device=DEV)
        cu, cub, sl = torch.empty(n + 1, **one), torch.empty(n + 1, **one), torch.empty(n, **one)
        req, lens, slots, left = (torch.empty(k, **one) for k in (T, T, T, 1))
        spd.paged_assign_slots(i32(new), prefix, rows, free, count, F, BS, 1, table, cu, cub, sl, req, lens, slots, left)
        mags = 2.0 ** (step - 2)
        fused = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * mags).to(BF16).to(DEV)
        s = dict(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:], wq=w, wk=w, cos_sin=cs, lens=lens, slots=slots,
                 kc=kc, vc=vc, ks=ks, vs=vs)
        before = {x: B.kept(s[x]) for x in CACHES}
        q = nan_like((T, Hq, D), BF16, DEV)
        out = nan_like((T, Hq, D), BF16, DEV)
        out2 = nan_like((T, Hq, D), BF16, DEV)
        ws = torch.empty(spd.prefill_attention_workspace_bytes(T, Hq, Hkv, D, n, NB), dtype=torch.uint8, device=DEV)
        ws2 = torch.empty(spd.decode_workspace_bytes(T, Hq, Hkv, D, NB), dtype=torch.uint8, device=DEV)

        def calls():
            spd.paged_norm_rope_store_block_scaled(*[s[x] for x in ("q", "k", "v", "wq", "wk", "cos_sin", "lens", "slots")], q,
                                                   kc, vc, ks, vs, 1e-6, False, BS)
            spd.paged_prefill_attention_block_scaled(q, kc, vc, ks, vs, table, rows, cu, sl, prefix, out, D ** -0.5, BS, ws)
            spd.paged_decode_attention_block_scaled(q, kc, vc, ks, vs, table, lens, req, out2, D ** -0.5, BS, ws2)

        if step % 2:
            saved = {x: s[x].clone() for x in CACHES}
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                calls()  # kernels are loaded before the capture
            torch.cuda.current_stream().wait_stream(side)
            for x in CACHES:
                s[x].view(torch.uint8).copy_(saved[x].view(torch.uint8))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
            for x in CACHES:
                s[x].view(torch.uint8).copy_(saved[x].view(torch.uint8))
            q.fill_(float("nan"))
            out.fill_(float("nan"))
            out2.fill_(float("nan"))
            graph.replay()
        else:
            calls()
        torch.cuda.synchronize()
        B.check_store(s, before, {x: B.kept(s[x]) for x in CACHES}, q, 1e-6, False, "step %d" % step)
        ref = B.attention(q, kc, vc, ks, vs, table, rows, cu, sl, prefix, D ** -0.5)
        B.check_attention(out, *ref, "prefill, step %d" % step)
        B.check_attention(out2, *ref, "decode, step %d" % step)
        lengths = [a + b for a, b in zip(lengths, new)]
        assert R.ints(sl).tolist() == lengths
        prefix, count = sl, left


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("K", [0, 3])
def test_graph_replays_with_new_scales(spd, which, K):
    s = attention_inputs([700, 300, 90], [4, 2, 1], 64, 8, 128, BF16, 41, K=K, pad=1)
    T, Hq, D = s["q"].shape
    out = nan_like((T, Hq, D), BF16, DEV)
    run = run_decode if which == "decode" else run_prefill
    if which == "decode":
        ws = torch.empty(spd.decode_workspace_bytes(T, Hq, 8, D, s["NB"]), dtype=torch.uint8, device=DEV)
        f = spd.paged_decode_attention_block_scaled if not K else spd.paged_sparse_decode_attention_block_scaled
        args = [s[n] for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "req")] + ([s["topk"]] if K else [])
    else:
        ws = torch.empty(spd.prefill_attention_workspace_bytes(T, Hq, 8, D, 3, s["NB"], s["topk"].shape[1] if K else 0),
                         dtype=torch.uint8, device=DEV)
        f = spd.paged_prefill_attention_block_scaled if not K else spd.paged_sparse_prefill_attention_block_scaled
        args = [s[n] for n in ("q", "kc", "vc", "ks", "vs", "table", "rows", "cu", "seq_lens", "prefix")] + (
            [s["topk"], s["bq"], s["cub"]] if K else [])
    run(spd, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(*args, out, s["sm"], BS, ws)
    for k in range(3):
        out.fill_(float("nan"))
        g = torch.Generator().manual_seed(k)
        for n in ("ks", "vs"):
            live = ~torch.isnan(s[n])
            s[n].copy_(torch.where(live, torch.exp2(torch.randint(-2, 3, s[n].shape, generator=g).float()).to(DEV), s[n]))
        s["q"].copy_(torch.randn(s["q"].shape, generator=g).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        ref = (B.decode(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["req"], s["sm"], s["topk"])
               if which == "decode" else
               B.attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["rows"], s["cu"], s["seq_lens"], s["prefix"],
                           s["sm"], s["topk"], s["bq"], s["cub"]))
        B.check_attention(out, *ref, "replay %d" % k)


def test_two_streams_at_once(spd):
    a = attention_inputs([2000, 300], [4, 2], 64, 8, 128, BF16, 42)
    b = attention_inputs([500, 1800], [60, 5], 64, 8, 128, BF16, 43)
    ref_a = B.decode(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["req"], a["sm"])
    ref_b = B.attention(b["q"], b["kc"], b["vc"], b["ks"], b["vs"], b["table"], b["rows"], b["cu"], b["seq_lens"], b["prefix"], b["sm"])
    oa, ob = nan_like(tuple(a["q"].shape), BF16, DEV), nan_like(tuple(b["q"].shape), BF16, DEV)
    wa = torch.empty(spd.decode_workspace_bytes(a["q"].shape[0], 64, 8, 128, a["NB"]), dtype=torch.uint8, device=DEV)
    wb = torch.empty(spd.prefill_attention_workspace_bytes(b["q"].shape[0], 64, 8, 128, 2, b["NB"]), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(8):
        spd.paged_decode_attention_block_scaled(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["req"], oa, a["sm"],
                                                BS, wa, stream=s1)
        spd.paged_prefill_attention_block_scaled(b["q"], b["kc"], b["vc"], b["ks"], b["vs"], b["table"], b["rows"], b["cu"],
                                                 b["seq_lens"], b["prefix"], ob, b["sm"], BS, wb, stream=s2)
    torch.cuda.synchronize()
    B.check_attention(oa, *ref_a, "decode")
    B.check_attention(ob, *ref_b, "prefill")


def test_both_ways_of_marshalling(spd, monkeypatch):
    from sparse_paged_decode_gb300 import binding

    if binding._fast is None:
        pytest.skip("the marshalling module is not built here")
    outs = []
    for compiled in (True, False):
        if not compiled:
            monkeypatch.setattr(binding, "_fast", None)
        s = store_inputs([(60, 100), (0, 3)], 8, 2, 128, 128, BF16, 11)
        got = [run_store(spd, s), s["kc"], s["vc"], s["ks"], s["vs"]]
        for K in (0, 3):
            a = attention_inputs([300, 200], [4, 2], 16, 2, 128, BF16, 44, K=K)
            got += [run_decode(spd, a), run_prefill(spd, a)]
        outs.append(digest(*got))
    assert outs[0] == outs[1]


# ------------------------------------------------- decode of single rows


def shared_selection(s, K, seed, kind="random"):
    """One selection for all kv heads: repeated ids, -1 and ids past the table among them."""
    g = torch.Generator().manual_seed(seed)
    T, NB = s["q"].shape[0], s["NB"]
    tk = torch.randint(-1, NB + 2, (1, T, K), generator=g).to(I32)
    if kind == "whole":  # every block, in an order of its own, some of them twice
        tk = torch.stack([torch.cat((torch.randperm(NB, generator=g), torch.randint(0, NB, (K,), generator=g)))[:K] for _ in range(T)])[None].to(I32)
    tk[0, ::5] = -1  # rows that select nothing
    s["topk"] = tk.to(DEV).expand(s["Hkv"], -1, -1)
    return s


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("heads", [(64, 8), (16, 2), (6, 2), (32, 2), (4, 4), (2, 2)])
@pytest.mark.parametrize("K,kind", [(1, "random"), (5, "random"), (12, "whole"), (40, "whole")])
def test_single_rows_with_a_shared_selection(spd, K, kind, heads, dt):
    s = attention_inputs([1300, 129, 700, 5, 1024, 256], [1, 1, 4, 1, 2, 1], *heads, 128, dt, 51, pad=2, general=True)
    check_decode(spd, shared_selection(s, K, 52, kind), (None, 1, 4), "K=%d %s" % (K, kind))


@pytest.mark.parametrize("K", [0, 9])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_single_rows_of_many_requests(spd, n, K):
    """Pieces that hold many rows, that end inside a row, and rows without keys among them."""
    r = random.Random(n)
    lengths = [r.choice((0, 1, 90, 128, 300, 1500)) if n > 1 else 3000 for _ in range(n)]
    s = attention_inputs(lengths, [1 if L else 0 for L in lengths], 16, 2, 128, BF16, 53, pad=3, NB=24)
    if K:
        shared_selection(s, K, 54)
    check_decode(spd, s, (None, 4), "%d requests" % n)


@pytest.mark.parametrize("heads", [(8, 2), (64, 64)])
def test_single_rows_over_long_page_tables(spd, heads):
    """Up to 1024 blocks, and pieces of more blocks than the kernel lists at a time (against 64 bits on the GPU)."""
    Hq, Hkv = heads
    D, NB, T = 128, 1024 if Hkv == 2 else 300, 3 if Hkv == 2 else 8
    g = torch.Generator(device=DEV).manual_seed(55)
    pool = NB + 3
    kc, vc = (torch.randn((pool * BS, Hkv, D), generator=g, device=DEV).mul_(m).to(E4M3) for m in (2.0, 60.0))
    ks, vs = (torch.exp2(torch.randint(-2, 3, (pool, Hkv), generator=g, device=DEV).float()) for _ in range(2))
    table = torch.randperm(pool, generator=g, device=DEV)[:NB].to(I32)[None].contiguous()
    lens = i32([NB * BS - 77 * i for i in range(T)])
    q = torch.randn((T, Hq, D), generator=g, device=DEV).to(BF16)
    out = nan_like((T, Hq, D), BF16, DEV)
    ws = torch.randint(0, 256, (spd.decode_workspace_bytes(T, Hq, Hkv, D, NB),), dtype=torch.uint8, device=DEV)
    old = spd.set_kernel_policy(3, 4)
    try:
        spd.paged_decode_attention_block_scaled(q, kc, vc, ks, vs, table, lens, i32([0] * T), out, D ** -0.5, BS, ws)
    finally:
        spd.set_kernel_policy(3, old)
    torch.cuda.synchronize()
    assert spd.workspace_status(ws) & 1 == 0
    G = Hq // Hkv
    for h in sorted({0, 1, Hkv // 2, Hkv - 1}):
        pages = table[0].long()
        k = (kc.view(pool, BS, Hkv, D)[pages, :, h].double() * ks[pages, h].double()[:, None, None]).view(-1, D)
        v = (vc.view(pool, BS, Hkv, D)[pages, :, h].double() * vs[pages, h].double()[:, None, None]).view(-1, D)
        for t in range(T):
            n = int(lens[t])
            z = q[t, h * G:(h + 1) * G].double() @ k[:n].T * D ** -0.5
            p = torch.softmax(z, -1)
            ref, A = p @ v[:n], p @ v[:n].abs()
            most = (p * vs[pages, h].double().repeat_interleave(BS)[:n]).amax(-1, keepdim=True)
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * A + n * 2.0 ** -22 * 448 * most
            assert bool(((out[t, h * G:(h + 1) * G].double() - ref).abs() <= tol).all()), (h, t)


@pytest.mark.parametrize("pol", [0, 4])
def test_single_rows_not_finite(spd, pol):
    """A NaN that a row reads shows in its dims (V) or its heads (K, q), and nowhere else."""
    s = attention_inputs([700, 300, 400], [1, 1, 1], 16, 2, 128, BF16, 56)
    t = s["table"][s["rows"].long()].long()
    s["vc"].view(torch.uint8)[t[0, 2] * BS + 5, 1, 17] = 0x7F
    s["kc"].view(torch.uint8)[t[1, 0] * BS + 9, 0, 3] = 0xFF
    s["q"][2, 5, 64] = float("inf")
    old = spd.set_kernel_policy(3, pol)
    try:
        out = run_decode(spd, s, None)
    finally:
        spd.set_kernel_policy(3, old)
    bad = torch.isnan(out.float())
    want = torch.zeros_like(bad)
    want[0, 8:, 17] = True
    want[1, :8] = True
    want[2, 5] = True
    assert torch.equal(bad, want)
