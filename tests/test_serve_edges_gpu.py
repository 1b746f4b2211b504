"""Serving-step calls on the GPU at the edges of their range: units of which a
tile takes nothing, heads that end inside a warp, infinities behind a join,
long page tables.  Definitions and tolerances are those of serve_ref.py."""
import numpy as np
import pytest
import torch

import serve_ref as R
from test_serve_gpu import BF16, BS, DEV, E4M3, F16, F32, I32, chunk_inputs, policy, run_chunk, run_store, store_inputs

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
