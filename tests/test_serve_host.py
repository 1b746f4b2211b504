"""Refusals of the serving-step calls on the host (no GPU needed): the error
code that the header documents, before any launch.  Descriptors carry fake
device addresses; a call that passes validation is only enqueued, so without
a GPU it reports SPD_ERR_CUDA."""
import pytest

import ctypes

from test_abi_host import (BF16, E4M3, F16, F32, I32, SPD_ERR_ALIASING, SPD_ERR_CUDA, SPD_ERR_INVALID_ARGUMENT,
                           SPD_ERR_UNSUPPORTED, SPD_ERR_WORKSPACE, SPD_OK, Fake, status)


def raw(fake):
    """The descriptor as the binding passes it to these calls."""
    return None if fake is None else ctypes.string_at(ctypes.addressof(fake.d), ctypes.sizeof(fake.d))


INVALID, UNSUPPORTED, ALIASING, WORKSPACE = SPD_ERR_INVALID_ARGUMENT, SPD_ERR_UNSUPPORTED, SPD_ERR_ALIASING, SPD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def spd():
    import torch

    if torch.cuda.is_available():
        pytest.skip("fake addresses: the calls that pass validation must not launch")
    from sparse_paged_decode_gb300 import binding

    return binding


def assign_call(spd, n_pages=64, block_size=128, bsq=4, **over):
    B, T = 3, 20
    t = dict(new=Fake((B,), I32), pre=Fake((B,), I32), sid=Fake((B,), I32), fp=Fake((30,), I32), fc=Fake((1,), I32),
             bt=Fake((4, 16), I32), cu=Fake((B + 1,), I32), cub=Fake((B + 1,), I32), sl=Fake((B,), I32),
             req=Fake((T,), I32), tl=Fake((T,), I32), slots=Fake((T,), I32), left=Fake((1,), I32))
    t.update(over)
    r = {k: raw(v) for k, v in t.items()}
    spd.lib.paged_assign_slots(r["new"], r["pre"], r["sid"], r["fp"], r["fc"], n_pages, block_size, bsq, r["bt"], r["cu"],
                               r["cub"], r["sl"], r["req"], r["tl"], r["slots"], r["left"], None)
    return status(spd)[0]


def test_assign_refusals(spd):
    assert assign_call(spd) in (SPD_OK, SPD_ERR_CUDA)
    assert assign_call(spd, block_size=64) == UNSUPPORTED
    assert assign_call(spd, bsq=0) == INVALID
    assert assign_call(spd, n_pages=-1) == UNSUPPORTED
    assert assign_call(spd, n_pages=1 << 24) == UNSUPPORTED
    assert assign_call(spd, pre=Fake((4,), I32)) == INVALID
    assert assign_call(spd, cu=Fake((3,), I32)) == INVALID
    assert assign_call(spd, slots=Fake((21,), I32)) == INVALID
    assert assign_call(spd, fc=Fake((2,), I32)) == INVALID
    assert assign_call(spd, left=None) == INVALID
    assert assign_call(spd, new=Fake((3,), F32)) == UNSUPPORTED
    assert assign_call(spd, bt=Fake((4, 1025), I32)) == UNSUPPORTED
    assert assign_call(spd, bt=Fake((4, 0), I32)) == UNSUPPORTED
    n = 8193
    assert assign_call(spd, new=Fake((n,), I32), pre=Fake((n,), I32), sid=Fake((n,), I32), sl=Fake((n,), I32),
                       cu=Fake((n + 1,), I32), cub=Fake((n + 1,), I32)) == UNSUPPORTED
    # an output over an input, over another output, over itself
    fc = Fake((1,), I32)
    assert assign_call(spd, fc=fc, left=Fake((1,), I32, addr=fc.d.data)) == ALIASING
    req = Fake((20,), I32)
    assert assign_call(spd, req=req, tl=Fake((20,), I32, addr=req.d.data + 40)) == ALIASING
    assert assign_call(spd, req=Fake((20,), I32, strides=(0,))) == INVALID
    assert assign_call(spd, bt=Fake((4, 16), I32, strides=(8, 1))) == ALIASING


def store_call(spd, T=5, Hq=8, Hkv=2, D=64, P=4, dt=BF16, cache=E4M3, eps=1e-6, block_size=128, ks=0.1, vs=0.1, **over):
    t = dict(q=Fake((T, Hq, D), dt), k=Fake((T, Hkv, D), dt), v=Fake((T, Hkv, D), dt), wq=Fake((D,), BF16),
             wk=Fake((D,), F32), cs=Fake((100, D), F32), tl=Fake((T,), I32), slots=Fake((T,), I32),
             qo=Fake((T, Hq, D), BF16), kc=Fake((P * 128, Hkv, D), cache), vc=Fake((P * 128, Hkv, D), cache))
    t.update(over)
    r = [raw(t[k]) for k in ("q", "k", "v", "wq", "wk", "cs", "tl", "slots", "qo", "kc", "vc")]
    spd.lib.paged_norm_rope_store(*r, eps, 0, block_size, ks, vs, None)
    return status(spd)[0]


def test_store_refusals(spd):
    ok = (SPD_OK, SPD_ERR_CUDA)
    assert store_call(spd) in ok
    assert store_call(spd, v=None, vc=None) in ok
    assert store_call(spd, wq=None, wk=None) in ok
    assert store_call(spd, cache=F32) in ok
    assert store_call(spd, T=0) == SPD_OK
    assert store_call(spd, v=None) == INVALID
    assert store_call(spd, vc=None) == INVALID
    assert store_call(spd, dt=E4M3) == UNSUPPORTED
    assert store_call(spd, k=Fake((5, 2, 64), F16)) == UNSUPPORTED
    assert store_call(spd, k=Fake((4, 2, 64), BF16)) == INVALID
    assert store_call(spd, kc=Fake((512, 2, 64), BF16)) == INVALID  # the caches' dtypes differ
    assert store_call(spd, kc=Fake((500, 2, 64), E4M3), vc=Fake((500, 2, 64), E4M3)) == INVALID
    assert store_call(spd, wq=Fake((32,), BF16)) == INVALID
    assert store_call(spd, wq=Fake((64,), E4M3)) == UNSUPPORTED
    assert store_call(spd, cs=Fake((100, 63), F32)) == UNSUPPORTED
    assert store_call(spd, cs=Fake((100, 66), F32)) == UNSUPPORTED
    assert store_call(spd, cs=Fake((100, 0), F32)) == UNSUPPORTED
    assert store_call(spd, cs=Fake((100, 64), BF16)) == UNSUPPORTED
    assert store_call(spd, D=512) == UNSUPPORTED
    assert store_call(spd, tl=Fake((6,), I32)) == INVALID
    assert store_call(spd, block_size=16) == UNSUPPORTED
    for bad in (float("nan"), float("inf"), -1.0):
        assert store_call(spd, eps=bad) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert store_call(spd, ks=bad) == INVALID
        assert store_call(spd, vs=bad) == INVALID
    q = Fake((5, 8, 64), BF16)
    assert store_call(spd, q=q, qo=Fake((5, 8, 64), BF16, addr=q.d.data)) == ALIASING
    kc = Fake((512, 2, 64), E4M3)
    assert store_call(spd, kc=kc, vc=Fake((512, 2, 64), E4M3, addr=kc.d.data)) == ALIASING
    # K and V interleaved slot by slot in one allocation are disjoint; shifted by half a row they are not
    both = Fake((512, 4, 64), E4M3)
    k_half = Fake((512, 2, 64), E4M3, strides=(256, 64, 1), addr=both.d.data)
    assert store_call(spd, kc=k_half, vc=Fake((512, 2, 64), E4M3, strides=(256, 64, 1), addr=both.d.data + 128)) in ok
    assert store_call(spd, kc=k_half, vc=Fake((512, 2, 64), E4M3, strides=(256, 64, 1), addr=both.d.data + 64)) == ALIASING


def chunk_call(spd, total_q=10, Hq=8, Hkv=2, D=64, B=2, NB=16, P=8, dt=BF16, cache=E4M3, sparse=True, K=4, n_rows=5, bsq=4,
               block_size=128, sm=0.1, ks=1.0, vs=1.0, short=0, shift=0, **over):
    t = dict(q=Fake((total_q, Hq, D), dt), k=Fake((P * 128, Hkv, D), cache), v=Fake((P * 128, Hkv, D), cache),
             bt=Fake((3, NB), I32), sid=Fake((B,), I32), cu=Fake((B + 1,), I32), sl=Fake((B,), I32), pre=Fake((B,), I32),
             tk=Fake((Hkv, n_rows, K), I32, strides=(0, K, 1)), cub=Fake((B + 1,), I32), out=Fake((total_q, Hq, D), BF16))
    t.update(over)
    r = {k: raw(v) for k, v in t.items() if k != "ws"}
    need = spd.lib.spd_prefill_attention_workspace_bytes(total_q, Hq, Hkv, D, B, NB, n_rows if sparse else 0)
    ws = Fake((max(need, 1) + 512,), E4M3)
    head = [r[k] for k in ("q", "k", "v", "bt", "sid", "cu", "sl", "pre")]
    tail = (sm, block_size, ks, vs, over.get("ws", ws.d.data) + shift, max(need - short, 0), None)
    if sparse:
        spd.lib.paged_sparse_prefill_attention(*head, r["tk"], bsq, r["cub"], r["out"], *tail)
    else:
        spd.lib.paged_prefill_attention(*head, r["out"], *tail)
    return status(spd)[0]


@pytest.mark.parametrize("sparse", [False, True])
def test_prefill_attention_refusals(spd, sparse):
    def call(**kw):
        return chunk_call(spd, sparse=sparse, **kw)

    ok = (SPD_OK, SPD_ERR_CUDA)
    assert call() in ok
    for D in (1, 96, 128, 256):
        for cache in (BF16, E4M3):
            for dt in (F32, F16, BF16):
                assert call(D=D, cache=cache, dt=dt) in ok
    assert call(total_q=0) == SPD_OK
    assert call(D=257) == UNSUPPORTED
    assert call(Hq=9) == UNSUPPORTED
    assert call(Hq=64, Hkv=2) == UNSUPPORTED
    assert call(dt=E4M3) == UNSUPPORTED
    assert call(cache=F16) == UNSUPPORTED
    assert call(v=Fake((1024, 2, 64), BF16)) == INVALID
    assert call(v=Fake((1152, 2, 64), E4M3)) == INVALID
    assert call(k=Fake((1000, 2, 64), E4M3), v=Fake((1000, 2, 64), E4M3)) == INVALID
    assert call(k=Fake((1024, 2, 64), E4M3, strides=(256, 128, 2))) == UNSUPPORTED
    assert call(bt=Fake((3, 1025), I32)) == UNSUPPORTED
    assert call(cu=Fake((2,), I32)) == INVALID
    assert call(sl=Fake((3,), I32)) == INVALID
    assert call(block_size=64) == UNSUPPORTED
    assert call(out=Fake((10, 8, 64), F32)) == UNSUPPORTED
    assert call(out=Fake((10, 8, 32), BF16)) == INVALID
    assert call(out=Fake((10, 8, 64), BF16, strides=(0, 64, 1))) == INVALID
    for bad in (float("nan"), float("inf")):
        assert call(sm=bad) == INVALID
        assert call(ks=bad) == INVALID
        assert call(vs=bad) == INVALID
    assert call(short=1) == WORKSPACE
    assert call(shift=64) == WORKSPACE
    q = Fake((10, 8, 64), BF16)
    assert call(q=q, out=Fake((10, 8, 64), BF16, addr=q.d.data + 128)) == ALIASING
    sl = Fake((2,), I32)
    assert call(sl=sl, ws=sl.d.data // 4096 * 4096) == ALIASING
    n = 8193
    assert call(B=n) == UNSUPPORTED
    if sparse:
        assert call(K=0) == INVALID
        assert call(bsq=0) == INVALID
        assert call(cub=Fake((2,), I32)) == INVALID
        assert call(tk=Fake((3, 5, 4), I32)) == INVALID
        assert call(tk=None) == INVALID
        assert call(tk=Fake((2, 5, 4), F32)) == UNSUPPORTED


def test_prefill_attention_workspace_sizes(spd):
    size = spd.lib.spd_prefill_attention_workspace_bytes
    base = size(64, 64, 8, 128, 4, 128, 0)
    assert base > 0 and size(64, 64, 8, 128, 4, 128, 100) >= base and size(4096, 64, 8, 128, 8, 128, 0) >= base
    for bad in ((-1, 8, 8, 64, 1, 4, 0), (1, 8, 0, 64, 1, 4, 0), (1, 9, 8, 64, 1, 4, 0), (1, 64, 2, 64, 1, 4, 0),
                (1, 8, 8, 257, 1, 4, 0), (1, 8, 8, 64, 8193, 4, 0), (1, 8, 8, 64, 1, 0, 0), (1, 8, 8, 64, 1, 1025, 0),
                (1, 8, 8, 64, 1, 4, -1), (1 << 30, 8, 8, 64, 1, 4, 0)):
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("compiled", [True, False])
def test_binding_refuses_what_is_not_on_the_gpu(spd, compiled, monkeypatch):
    """Both ways that the binding marshals, the compiled module and the
    Python descriptors, refuse alike."""
    import torch

    if compiled and spd._fast is None:
        pytest.skip("the marshalling module is not built here")
    if not compiled:
        monkeypatch.setattr(spd, "_fast", None)

    x = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        spd.paged_assign_slots(*[x] * 5, 8, 128, 1, *[x] * 8)
    with pytest.raises(ValueError):
        spd.paged_norm_rope_store(*[x] * 11, 1e-6, False, 128, 1.0, 1.0, stream=0)
    with pytest.raises(TypeError):
        spd.paged_prefill_attention(*[x.double()] * 9, 1.0, 128, 1.0, 1.0, None, stream=0)
    with pytest.raises(TypeError):
        spd.paged_prefill_attention(*["x"] * 9, 1.0, 128, 1.0, 1.0, None, stream=0)
    with pytest.raises(ValueError):
        spd.paged_prefill_attention(*[torch.zeros((0,) * 5)] * 9, 1.0, 128, 1.0, 1.0, None, stream=0)
    with pytest.raises(TypeError):
        spd.paged_prefill_attention(*[torch.zeros(0)] * 9, 1.0, 128, 1.0, 1.0, x, stream=0)
    with pytest.raises(spd.SpdError) as e:  # past the binding: refused by the library
        spd.paged_prefill_attention(*[torch.zeros(0)] * 9, 1.0, 128, 1.0, 1.0, None, stream=0)
    assert e.value.code == INVALID
