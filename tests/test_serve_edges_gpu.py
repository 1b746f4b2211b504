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
