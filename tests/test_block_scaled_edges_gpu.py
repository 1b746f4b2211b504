"""Block-scaled calls where a mistake would be rare or silent, against the 64-bit
definitions and tolerances of block_scaled_ref.py."""
import pytest
import torch

from test_block_scaled_gpu import (BF16, BS, DEV, E4M3, F16, attention_inputs, check_decode, check_prefill, check_store,
                                   run_decode, run_prefill, run_store, shared_selection, spd, store_inputs)  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("heads", [(16, 2), (32, 2)])
@pytest.mark.parametrize("K", [0, 1])
def test_pieces_of_one_page_repeat_themselves(spd, K, heads, dt):  # noqa: F811
    """Every row's only page raises the offset and ends its piece: the maxima of its
    warps are read just before their sums are written.  A quarter of the keys (one
    warp's) carries the weight, so a sum taken for a maximum would show."""
    n = 160
    s = attention_inputs([1 + 37 * i % 128 if not K else 129 + 37 * i % 512 for i in range(n)], [1] * n, *heads, 128, dt, 81)
    if K:
        shared_selection(s, K, 82)
    t = s["table"][s["rows"].long()].long()
    kc = s["kc"].view(torch.uint8).view(-1, BS, heads[1], 128)
    for w in range(4):
        page, keys = t[w::4, 0], slice(32 * w, 32 * w + 32)
        kc[page, keys] = (kc[page, keys].view(E4M3).float() * 8).clamp(-448, 448).to(E4M3).view(torch.uint8)
    check_decode(spd, s, (None, 4), "one page")
    first = run_decode(spd, s, 4)
    ws = torch.zeros((spd.decode_workspace_bytes(n, heads[0], heads[1], 128, s["NB"]),), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(first)
    f = spd.paged_decode_attention_block_scaled if s["topk"] is None else spd.paged_sparse_decode_attention_block_scaled
    ins = [s[x] for x in ("q", "kc", "vc", "ks", "vs", "table", "lens", "req")] + ([s["topk"]] if K else [])
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(400):
        f(*ins, out, s["sm"], BS, ws)
        differ += (out.view(torch.int16) != first.view(torch.int16)).sum()
    assert int(differ) == 0


# ------------------------------------------------ V scales far apart in a row
#
# Both ends of the range, 2^-64 and 2^64, in one row.  The keys of the low pages
# add next to nothing to the row's products and most of its softmax sum: without
# them the output would be up to (low + high pages) / (high pages) times as large,
# where the bound allows it to be off by 2^-7.

ORDERS = {"low first": lambda j, n: j < n - 2, "high first": lambda j, n: j >= 2, "one low": lambda j, n: j == n // 2,
          "one high": lambda j, n: j != n // 2, "in turn": lambda j, n: j % 2 == 0}


def far_apart(lengths, new, Hq, Hkv, D, dt, seed, order, level, low=-64, high=64, **kw):
    """Requests whose pages have V scales of 2^low or 2^high; the logits of the low
    pages lie level / sqrt(D) above the others'."""
    s = attention_inputs(lengths, new, Hq, Hkv, D, dt, seed, **kw)
    s["q"][:, :, 0] = 1.0
    kc, t = s["kc"].view(torch.uint8).view(-1, BS, Hkv, D), s["table"][s["rows"].long()].long()
    code = int(torch.tensor(float(level)).to(E4M3).view(torch.uint8))
    for b, L in enumerate(lengths):
        n = -(-L // BS)
        for j in range(n):
            is_low = ORDERS[order](j, n)
            s["vs"][t[b, j]] = 2.0 ** (low if is_low else high)
            s["ks"][t[b, j]] = 1.0
            kc[t[b, j], :L - j * BS, :, 0] = code if is_low else 0
    return s


@pytest.mark.parametrize("level", [-32, 0, 96])
@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("heads", [(16, 2), (32, 2), (9, 3)])
def test_decode_v_scales_at_both_ends(spd, heads, order, level):  # noqa: F811
    for K in (0, 9):
        s = far_apart([2300, 130, 1000, 2000], [1, 2, 16, 1], *heads, 128, BF16, 83, order, level, K=K)
        check_decode(spd, s, (None, 1, 2, 3, 4), "%s, K=%d" % (order, K))


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("order", list(ORDERS))
def test_decode_v_scales_at_both_ends_of_single_rows(spd, order, dt):  # noqa: F811
    s = far_apart([6000, 257, 3001], [1, 1, 1], 8, 2, 128, dt, 84, order, 0)  # rows in many pieces
    check_decode(spd, s, (None, 2, 3, 4), order)


@pytest.mark.parametrize("level", [-32, 0, 96])
@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("kind", [(128, BF16), (128, F16), (64, BF16)], ids=["terms", "f16", "wide64"])
def test_prefill_v_scales_at_both_ends(spd, kind, order, level):  # noqa: F811
    D, dt = kind
    for K in (0, 9):
        s = far_apart([2300, 130, 1000, 3000], [3, 2, 150, 20], 16, 2, D, dt, 85, order, level, K=K, bq=16)
        check_prefill(spd, s, (None, 1), "%s, K=%d" % (order, K))


@pytest.mark.parametrize("apart", [(-33, 64), (-32, 64), (-31, 64), (-64, 40), (-64, 63)])
def test_v_scales_around_the_low_ones(spd, apart):  # noqa: F811
    """Either side of 2^-32, below which a page adds its weights apart from its products."""
    for order in ("low first", "one high"):
        s = far_apart([2300, 130], [1, 16], 16, 2, 128, BF16, 86, order, 32, *apart)
        check_decode(spd, s, (None, 2, 3, 4), "decode, " + order)
        check_prefill(spd, s, (None,), "prefill, " + order)


# ------------------------------------------------------- long page tables


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("K", [0, 5])
@pytest.mark.parametrize("new", [(1, 1), (3, 2), (16, 16)], ids=["single", "drafts", "wide"])
def test_decode_over_long_page_tables_by_default(spd, new, K, dt):  # noqa: F811
    """More than 256 blocks, whatever the rows of a request: a tensor-core kernel (two
    launches), not the general one."""
    s = attention_inputs([700, 1290], list(new), 16, 2, 128, dt, 87, NB=300)
    if K:
        shared_selection(s, K, 88, "whole")
    before = spd.launch_count()
    run_decode(spd, s)
    assert spd.launch_count() - before == 2
    check_decode(spd, s, (None,), "long table")


# ------------------------------------------- K and V parts of one allocation


@pytest.mark.parametrize("cache", ["slots", "heads"])
@pytest.mark.parametrize("scale", ["rows", "pairs"])
@pytest.mark.parametrize("dt", [BF16, torch.float32], ids=["vector", "general"])
def test_store_and_attention_over_parts_of_one_allocation(spd, dt, scale, cache):  # noqa: F811
    """Scales [P, 2, Hkv] or [P, Hkv, 2], caches [slots, 2, Hkv, D] or [slots, Hkv, 2, D]: K and V as views."""
    s = store_inputs([(60, 100), (0, 30), (126, 9)], 8, 2, 128, 128, dt, 89)
    at = {"slots": 1, "heads": 2}[cache]
    both = torch.stack((s["kc"].view(torch.uint8), s["vc"].view(torch.uint8)), at).view(E4M3)
    s["kc"], s["vc"] = both.select(at, 0), both.select(at, 1)
    both = torch.stack((s["ks"], s["vs"]), {"rows": 1, "pairs": 2}[scale])
    s["ks"], s["vs"] = both.select({"rows": 1, "pairs": 2}[scale], 0), both.select({"rows": 1, "pairs": 2}[scale], 1)
    check_store(spd, s, "%s, %s" % (scale, cache))
    s["ks"].fill_(2.0 ** -5)  # logits of a few units
    a = attention_inputs([300, 70], [3, 2], 8, 2, 128, BF16, 90)
    a.update({x: s[x] for x in ("kc", "vc", "ks", "vs")}, table=a["table"].clamp(0, s["ks"].shape[0] - 1))
    check_decode(spd, a, (None, 1), "decode")
    check_prefill(spd, a, (None, 1), "prefill")


# ----------------------------------------------------------------- repeats


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("K", [0, 7])
def test_attention_repeats_itself(spd, K, which):  # noqa: F811
    """Which CTA takes a unit and which joins a row's pieces changes from call to call; no bit of the output does."""
    new = [1, 4, 16, 1, 8, 2] if which == "decode" else [100, 4, 333, 1, 64, 2]
    s = attention_inputs([4000, 1300, 2500, 700, 3100, 129], new, 64, 8, 128, BF16, 91, K=K, bq=16 if which == "prefill" else 1, wild=6)
    if K and which == "decode":
        shared_selection(s, K, 92)
    run = run_decode if which == "decode" else run_prefill
    for pol in (None, 2, 3, 4) if which == "decode" else (None,):
        first = run(spd, s, pol).view(torch.int16)
        for _ in range(25):
            assert torch.equal(run(spd, s, pol).view(torch.int16), first), pol


def test_store_repeats_itself(spd):  # noqa: F811
    def once():
        s = store_inputs([(p, 2 + p % 150) for p in range(0, 1270, 29)], 8, 4, 128, 128, BF16, 93, pad=5)
        out = run_store(spd, s)
        return [x.view(torch.uint8) for x in (out, s["kc"], s["vc"], s["ks"], s["vs"])]

    first = once()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(once(), first))
