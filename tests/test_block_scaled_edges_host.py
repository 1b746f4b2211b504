"""Calls of the block-scaled and static decode attention on the host (no GPU
needed) that a user may make and that once ended the process or were refused."""
import itertools
import random

import pytest

import test_serve_host
from test_abi_host import BF16, E4M3, F32, I32, SPD_ERR_CUDA, SPD_OK, Fake, status
from test_block_scaled_host import store_call
from test_serve_host import ALIASING, raw, spd  # noqa: F401 (fixture)


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


# strides of K's and V's half of one allocation, and the distance between them, in elements
SCALES = {"rows of 2 Hkv": ((8, 1), 4), "pairs": ((8, 2), 1), "heads first": ((2, 10), 1), "pages of both": ((2, 20), 1)}
CACHES = {"slots of 2 Hkv": ((512, 64, 1), 256), "heads of 2 D": ((512, 128, 1), 64), "pages of one": ((512, 64, 1), -256)}


@pytest.mark.parametrize("layout", list(SCALES))
def test_store_takes_scales_side_by_side(spd, layout):  # noqa: F811
    strides, apart = SCALES[layout]
    ks = Fake((5, 4), F32, strides=strides)
    for a, b in ((0, apart), (apart, 0)):
        kw = dict(Hkv=4, P=5, ks=Fake((5, 4), F32, strides=strides, addr=ks.d.data + 4 * a),
                  vs=Fake((5, 4), F32, strides=strides, addr=ks.d.data + 4 * b))
        assert store_call(spd, **kw) in (SPD_OK, SPD_ERR_CUDA)
    # the same cells, and a page on
    for shift in (0, strides[0], -strides[1]):
        assert store_call(spd, Hkv=4, P=5, ks=ks, vs=Fake((5, 4), F32, strides=strides, addr=ks.d.data + 4 * shift)) == ALIASING
    # other strides: not looked into
    assert store_call(spd, Hkv=4, P=5, ks=ks, vs=Fake((5, 4), F32, strides=(4, 1), addr=ks.d.data + 4)) == ALIASING


@pytest.mark.parametrize("block", [False, True], ids=["static", "block-scaled"])
@pytest.mark.parametrize("layout", list(CACHES))
def test_store_takes_caches_side_by_side(spd, layout, block):  # noqa: F811
    strides, apart = CACHES[layout]
    call = store_call if block else test_serve_host.store_call
    room = Fake((2048, 4, 64), E4M3)  # addresses that no other operand has
    kc = Fake((512, 4, 64), E4M3, strides=strides, addr=room.d.data + 4096)

    def other(shift):
        return call(spd, Hkv=4, kc=kc, vc=Fake((512, 4, 64), E4M3, strides=strides, addr=kc.d.data + shift))

    assert other(apart) in (SPD_OK, SPD_ERR_CUDA)
    for shift in (0, 32, 2 * strides[1], strides[0], apart + 1, apart - 1):
        assert other(shift) == ALIASING


def test_side_by_side_is_exact(spd):  # noqa: F811
    """Random nested layouts and distances: refused where two cells are one, and only there."""
    r = random.Random(9)
    seen = {True: 0, False: 0}
    for _ in range(400):
        P, Hkv = r.randint(1, 4), r.choice((1, 2, 3))
        order, strides, span = r.sample((0, 1), 2), [0, 0], 1
        for d in order:
            strides[d] = span + r.randint(0, 3)
            span = strides[d] * ((P, Hkv)[d] - 1) + span
        apart = r.randint(-span - 1, span + 1)
        cells = {i * strides[0] + j * strides[1] for i, j in itertools.product(range(P), range(Hkv))}
        meet = any(c + apart in cells for c in cells)
        ks = Fake((P, Hkv), F32, strides=tuple(strides), addr=(1 << 45))
        vs = Fake((P, Hkv), F32, strides=tuple(strides), addr=(1 << 45) + 4 * apart)
        got = store_call(spd, Hq=Hkv, Hkv=Hkv, P=P, ks=ks, vs=vs)
        assert (got == ALIASING) == meet, (P, Hkv, strides, apart)
        assert meet or got in (SPD_OK, SPD_ERR_CUDA)
        seen[meet] += 1
    assert min(seen.values()) > 100
