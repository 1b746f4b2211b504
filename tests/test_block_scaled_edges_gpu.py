"""Block-scaled calls where a mistake would be rare or silent, against the 64-bit
definitions and tolerances of block_scaled_ref.py."""
import pytest
import torch

from test_block_scaled_gpu import (BF16, BS, DEV, E4M3, F16, attention_inputs, check_decode, run_decode, shared_selection,
                                   spd)  # noqa: F401 (fixture)

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
