"""Refusals of the block-scaled calls on the host (no GPU needed), as in
test_serve_host.py: the error code that the header documents, before any launch."""
import math

import pytest

from test_abi_host import BF16, E4M3, F16, F32, I32, SPD_ERR_CUDA, SPD_OK, Fake, status
from test_serve_host import ALIASING, INVALID, UNSUPPORTED, WORKSPACE, raw, spd  # noqa: F401 (fixture)

OK = (SPD_OK, SPD_ERR_CUDA)


def store_call(spd, T=5, Hq=8, Hkv=2, D=64, P=4, dt=BF16, cache=E4M3, eps=1e-6, block_size=128, **over):  # noqa: F811
    t = dict(q=Fake((T, Hq, D), dt), k=Fake((T, Hkv, D), dt), v=Fake((T, Hkv, D), dt), wq=Fake((D,), BF16),
             wk=Fake((D,), F32), cs=Fake((100, D), F32), tl=Fake((T,), I32), slots=Fake((T,), I32),
             qo=Fake((T, Hq, D), BF16), kc=Fake((P * 128, Hkv, D), cache), vc=Fake((P * 128, Hkv, D), cache),
             ks=Fake((P, Hkv), F32), vs=Fake((P, Hkv), F32))
    t.update(over)
    r = [raw(t[k]) for k in ("q", "k", "v", "wq", "wk", "cs", "tl", "slots", "qo", "kc", "vc", "ks", "vs")]
    spd.lib.paged_norm_rope_store_block_scaled(*r, eps, 0, block_size, None)
    return status(spd)[0]


def test_store_refusals(spd):  # noqa: F811
    def call(**kw):
        return store_call(spd, **kw)

    for dt in (F32, BF16, F16):
        for D in (2, 64, 96, 128, 256):
            assert call(dt=dt, D=D) in OK
    assert call(wq=None, wk=None) in OK
    assert call(T=0) == SPD_OK
    assert call(v=None, vc=None) == INVALID  # both caches are appended to
    assert call(v=None) == INVALID
    assert call(vc=None) == INVALID
    assert call(ks=None) == INVALID
    assert call(vs=None) == INVALID
    assert call(cache=BF16) == UNSUPPORTED
    assert call(cache=F32) == UNSUPPORTED
    assert call(vc=Fake((512, 2, 64), BF16)) == INVALID
    assert call(ks=Fake((4, 2), BF16)) == UNSUPPORTED
    assert call(ks=Fake((5, 2), F32)) == INVALID
    assert call(vs=Fake((4, 1), F32)) == INVALID
    assert call(vs=Fake((8,), F32)) == INVALID
    assert call(vs=Fake((4, 2), F32, strides=(0, 1))) == INVALID  # scales are written: no broadcast
    assert call(vs=Fake((4, 2), F32, strides=(1, 1))) == ALIASING
    assert call(vs=Fake((4, 2), F32, strides=(1, 4))) in OK
    ks = Fake((4, 2), F32)
    assert call(ks=ks, vs=Fake((4, 2), F32, addr=ks.d.data)) == ALIASING
    kc = Fake((512, 2, 64), E4M3)
    assert call(kc=kc, vs=Fake((4, 2), F32, addr=kc.d.data + 1024)) == ALIASING
    tl = Fake((5,), I32)
    assert call(tl=tl, ks=Fake((4, 2), F32, addr=tl.d.data)) == ALIASING
    qo = Fake((5, 8, 64), BF16)
    assert call(qo=qo, ks=Fake((4, 2), F32, addr=qo.d.data)) == ALIASING
    assert call(ks=Fake((4, 2), F32, addr=(1 << 40) + 2)) == INVALID  # not aligned to an element
    assert call(D=512) == UNSUPPORTED
    assert call(block_size=64) == UNSUPPORTED
    assert call(slots=Fake((6,), I32)) == INVALID
    assert call(kc=Fake((500, 2, 64), E4M3), vc=Fake((500, 2, 64), E4M3)) == INVALID
    for bad in (float("nan"), math.inf, -1.0):
        assert call(eps=bad) == INVALID


def attention_call(spd, which, sparse, T=6, Hq=8, Hkv=2, D=128, B=2, NB=16, P=8, dt=BF16, cache=E4M3, K=4, bq=1,  # noqa: F811
                   block_size=128, sm=0.1, short=0, shift=0, **over):
    t = dict(q=Fake((T, Hq, D), dt), k=Fake((P * 128, Hkv, D), cache), v=Fake((P * 128, Hkv, D), cache),
             ks=Fake((P, Hkv), F32), vs=Fake((P, Hkv), F32), bt=Fake((3, NB), I32), lens=Fake((T,), I32), req=Fake((T,), I32),
             sid=Fake((B,), I32), cu=Fake((B + 1,), I32), sl=Fake((B,), I32), pre=Fake((B,), I32),
             tk=Fake((Hkv, T, K), I32, strides=(0, K, 1)), cub=Fake((B + 1,), I32), out=Fake((T, Hq, D), BF16))
    t.update(over)
    r = {k: raw(v) for k, v in t.items() if k != "ws"}
    if which == "decode":
        need = spd.lib.spd_decode_workspace_bytes(T, Hq, Hkv, D, NB, 128)
    else:
        need = spd.lib.spd_prefill_attention_workspace_bytes(T, Hq, Hkv, D, B, NB, T if sparse else 0)
    ws = Fake((max(need, 1) + 512,), E4M3)
    head = [r[k] for k in ("q", "k", "v", "ks", "vs", "bt")]
    tail = (sm, block_size, over.get("ws", ws.d.data) + shift, max(need - short, 0), None)
    if which == "decode":
        f = spd.lib.paged_sparse_decode_attention_block_scaled if sparse else spd.lib.paged_decode_attention_block_scaled
        f(*head, r["lens"], r["req"], *([r["tk"]] if sparse else []), r["out"], *tail)
    else:
        f = spd.lib.paged_sparse_prefill_attention_block_scaled if sparse else spd.lib.paged_prefill_attention_block_scaled
        f(*head, r["sid"], r["cu"], r["sl"], r["pre"], *([r["tk"], bq, r["cub"]] if sparse else []), r["out"], *tail)
    return status(spd)[0]


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_attention_refusals(spd, which, sparse):  # noqa: F811
    def call(**kw):
        return attention_call(spd, which, sparse, **kw)

    for D in (1, 64, 96, 128, 256):
        for dt in (F32, F16, BF16):
            assert call(D=D, dt=dt) in OK
    assert call(T=0) == SPD_OK
    assert call(P=0) in OK
    for name in ("k", "v", "ks", "vs", "bt", "out"):
        assert call(**{name: None}) == INVALID
    assert call(cache=BF16) == UNSUPPORTED
    assert call(cache=F16) == UNSUPPORTED
    assert call(v=Fake((1024, 2, 128), BF16)) in (INVALID, UNSUPPORTED)
    assert call(ks=Fake((8, 2), F16)) == UNSUPPORTED
    assert call(ks=Fake((7, 2), F32)) == INVALID
    assert call(vs=Fake((8, 3), F32)) == INVALID
    assert call(vs=Fake((16,), F32)) == INVALID
    assert call(vs=Fake((8, 2), F32, strides=(0, 0))) in OK  # an input may be broadcast
    vs = Fake((8, 2), F32)
    assert call(vs=vs, out=Fake((6, 8, 128), BF16, addr=vs.d.data)) == ALIASING
    if which == "prefill":
        assert call(vs=vs, ws=vs.d.data // 4096 * 4096) == ALIASING
    for bad in (float("nan"), math.inf):
        assert call(sm=bad) == INVALID
    assert call(block_size=64) == UNSUPPORTED
    assert call(D=257) == UNSUPPORTED
    assert call(Hq=9) == UNSUPPORTED
    assert call(Hq=64, Hkv=2) == UNSUPPORTED
    assert call(short=1) == WORKSPACE
    assert call(shift=64) == WORKSPACE
    if sparse:
        assert call(tk=None) == INVALID
        assert call(K=0) == INVALID
        assert call(tk=Fake((3, 6, 4), I32)) == INVALID


@pytest.mark.parametrize("compiled", [True, False])
def test_binding_refuses_what_is_not_on_the_gpu(spd, compiled, monkeypatch):  # noqa: F811
    import torch

    if compiled and spd._fast is None:
        pytest.skip("the marshalling module is not built here")
    if not compiled:
        monkeypatch.setattr(spd, "_fast", None)
    x, none = torch.zeros(3, dtype=torch.int32), torch.zeros(0)
    with pytest.raises(ValueError):
        spd.paged_norm_rope_store_block_scaled(*[x] * 13, 1e-6, False, 128, stream=0)
    with pytest.raises(ValueError):
        spd.paged_decode_attention_block_scaled(*[x] * 9, 1.0, 128, None, stream=0)
    with pytest.raises(TypeError):
        spd.paged_sparse_decode_attention_block_scaled(*[x.double()] * 10, 1.0, 128, None, stream=0)
    with pytest.raises(TypeError):
        spd.paged_prefill_attention_block_scaled(*["x"] * 11, 1.0, 128, None, stream=0)
    with pytest.raises(TypeError):
        spd.paged_sparse_prefill_attention_block_scaled(*[none] * 11, 1, none, none, 1.0, 128, x, stream=0)
    for f, n in ((spd.paged_norm_rope_store_block_scaled, 13), (spd.paged_decode_attention_block_scaled, 9)):
        with pytest.raises(spd.SpdError) as e:  # past the binding: refused by the library
            f(*[none] * n, *((1e-6, False, 128) if n == 13 else (1.0, 128, None)), stream=0)
        assert e.value.code == INVALID
