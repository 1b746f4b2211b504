"""Calls of the block-scaled and static decode attention on the host (no GPU
needed) that a user may make and that once ended the process or were refused."""
import pytest

from test_abi_host import BF16, E4M3, F32, I32, SPD_OK, Fake, status
from test_serve_host import raw, spd  # noqa: F401 (fixture)


@pytest.mark.parametrize("ws", [False, True], ids=["no workspace", "workspace"])
@pytest.mark.parametrize("policy", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("block", [False, True], ids=["static", "block-scaled"])
def test_decode_without_query_heads(spd, block, sparse, policy, ws):  # noqa: F811
    """q [T, 0, D] as torch lays it out: nothing to write, as with no rows."""
    T, Hkv, D, K = 6, 2, 128, 4
    empty = Fake((T, 0, D), BF16, strides=(D, D, 1))
    cache, tk = Fake((1024, Hkv, D), E4M3), Fake((Hkv, T, K), I32, strides=(0, K, 1))
    tensors = [empty, cache, cache, *([Fake((8, Hkv), F32), Fake((8, Hkv), F32)] if block else []), Fake((3, 16), I32),
               Fake((T,), I32), Fake((T,), I32), *([tk] if sparse else []), empty]
    args = [raw(x) if block else x.ref() for x in tensors] + [0.1, 128, *([] if block else [1.0, 1.0])]
    space = Fake((1 << 20,), E4M3)
    name = ("paged_sparse_decode_attention" if sparse else "paged_decode_attention") + ("_block_scaled" if block else "")
    old = spd.lib.spd_set_kernel_policy(3, policy)
    try:
        getattr(spd.lib, name)(*args, *([space.d.data, 1 << 20] if ws else [None, 0]), None)
    finally:
        spd.lib.spd_set_kernel_policy(3, old)
    assert status(spd)[0] == SPD_OK
