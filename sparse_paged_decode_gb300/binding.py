"""Thin ctypes binding of libspd.so: torch tensors in, C ABI call, error check.

Argument marshalling only -- every step of every call runs in the CUDA
library.  Importing this module loads ``libspd.so`` (built in-tree by
``sparse_paged_decode_gb300.build``) and raises if it is missing: there is no
CPU or PyTorch fallback.  Each function enqueues on the current torch CUDA
stream unless a stream is given, returns None, and raises ``SpdError`` when
the library rejects the call (see ``include/spd.h``).
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

from .build import LIB_PATH

__all__ = [
    "SpdError",
    "msa_block_score",
    "msa_select_topk",
    "paged_sparse_decode_attention",
    "paged_decode_attention",
    "paged_sparse_decode_attention_noalloc",
    "attention_sdpa",
    "msa_prefill_block_score",
    "prefill_workspace_bytes",
    "paged_assign_slots",
    "paged_norm_rope_store",
    "paged_prefill_attention",
    "paged_sparse_prefill_attention",
    "paged_norm_rope_store_block_scaled",
    "paged_decode_attention_block_scaled",
    "paged_sparse_decode_attention_block_scaled",
    "paged_prefill_attention_block_scaled",
    "paged_sparse_prefill_attention_block_scaled",
    "prefill_attention_workspace_bytes",
    "decode_workspace_bytes",
    "launch_count",
    "set_attention_kernel",
    "set_kernel_policy",
    "workspace_status",
    "library_path",
    "lib",
]

SPD_F32, SPD_BF16, SPD_F16, SPD_E4M3, SPD_I32 = 0, 1, 2, 3, 4
_DTYPES = {
    torch.float32: SPD_F32,
    torch.bfloat16: SPD_BF16,
    torch.float16: SPD_F16,
    torch.float8_e4m3fn: SPD_E4M3,
    torch.int32: SPD_I32,
}


class SpdError(RuntimeError):
    """A call rejected by libspd (validation failure or launch error)."""

    def __init__(self, code: int, msg: str):
        super().__init__("spd error %d: %s" % (code, msg))
        self.code = code


class SpdTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("ndim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * 4),
        ("stride", ctypes.c_int64 * 4),
    ]


def library_path() -> str:
    return LIB_PATH


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "libspd.so is not built (%s); run `python -m sparse_paged_decode_gb300.build` "
            "or __graft_entry__.build() -- there is no fallback implementation" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(SpdTensor)
    vp, f32, i32, sz = ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_size_t
    L.msa_block_score.argtypes = [P, P, P, P, P, i32, P, f32, vp]
    L.msa_block_score.restype = None
    L.msa_select_topk.argtypes = [P, P, vp]
    L.msa_select_topk.restype = None
    L.paged_sparse_decode_attention.argtypes = [P, P, P, P, P, P, P, P, f32, i32, f32, f32, vp, sz, vp]
    L.paged_sparse_decode_attention.restype = None
    L.paged_sparse_decode_attention_noalloc.argtypes = [P, P, P, P, P, P, P, P, f32, i32, f32, f32, vp]
    L.paged_sparse_decode_attention_noalloc.restype = None
    L.paged_decode_attention.argtypes = [P, P, P, P, P, P, P, f32, i32, f32, f32, vp, sz, vp]
    L.paged_decode_attention.restype = None
    L.msa_prefill_block_score.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, f32, P, P, vp, sz, vp]
    L.msa_prefill_block_score.restype = None
    L.spd_prefill_workspace_bytes.argtypes = [ctypes.c_int64] * 3
    L.spd_prefill_workspace_bytes.restype = sz
    # the serving-step calls take their descriptors as packed bytes (_pack)
    B = ctypes.c_char_p
    L.paged_assign_slots.argtypes = [B] * 5 + [i32] * 3 + [B] * 8 + [vp]
    L.paged_assign_slots.restype = None
    L.paged_norm_rope_store.argtypes = [B] * 11 + [f32, i32, i32, f32, f32, vp]
    L.paged_norm_rope_store.restype = None
    L.paged_prefill_attention.argtypes = [B] * 9 + [f32, i32, f32, f32, vp, sz, vp]
    L.paged_prefill_attention.restype = None
    L.paged_sparse_prefill_attention.argtypes = [B] * 9 + [i32, B, B, f32, i32, f32, f32, vp, sz, vp]
    L.paged_sparse_prefill_attention.restype = None
    L.paged_norm_rope_store_block_scaled.argtypes = [B] * 13 + [f32, i32, i32, vp]
    L.paged_norm_rope_store_block_scaled.restype = None
    L.paged_decode_attention_block_scaled.argtypes = [B] * 9 + [f32, i32, vp, sz, vp]
    L.paged_decode_attention_block_scaled.restype = None
    L.paged_sparse_decode_attention_block_scaled.argtypes = [B] * 10 + [f32, i32, vp, sz, vp]
    L.paged_sparse_decode_attention_block_scaled.restype = None
    L.paged_prefill_attention_block_scaled.argtypes = [B] * 11 + [f32, i32, vp, sz, vp]
    L.paged_prefill_attention_block_scaled.restype = None
    L.paged_sparse_prefill_attention_block_scaled.argtypes = [B] * 11 + [i32, B, B, f32, i32, vp, sz, vp]
    L.paged_sparse_prefill_attention_block_scaled.restype = None
    L.spd_prefill_attention_workspace_bytes.argtypes = [ctypes.c_int64] * 7
    L.spd_prefill_attention_workspace_bytes.restype = sz
    L.attention_sdpa.argtypes = [P, P, P, P, f32, i32, vp]
    L.attention_sdpa.restype = None
    L.spd_decode_workspace_bytes.argtypes = [ctypes.c_int64] * 5 + [i32]
    L.spd_decode_workspace_bytes.restype = sz
    L.spd_last_error.argtypes = [ctypes.c_char_p, sz]
    L.spd_last_error.restype = ctypes.c_int
    L.spd_set_attention_kernel.argtypes = [ctypes.c_int]
    L.spd_set_attention_kernel.restype = ctypes.c_int
    L.spd_set_kernel_policy.argtypes = [ctypes.c_int, ctypes.c_int]
    L.spd_set_kernel_policy.restype = ctypes.c_int
    L.spd_workspace_status.argtypes = [vp, vp]
    L.spd_workspace_status.restype = ctypes.c_int
    L.spd_launch_count.argtypes = []
    L.spd_launch_count.restype = ctypes.c_uint64
    L.spd_version.argtypes = []
    L.spd_version.restype = ctypes.c_char_p
    return L


lib = _load()


def _desc(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DTYPES:
        raise TypeError("%s: dtype %s is not supported by libspd" % (name, t.dtype))
    if t.numel() > 0 and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() > 4:
        raise ValueError("%s has more than 4 dims" % name)
    d = SpdTensor()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _DTYPES[t.dtype]
    d.ndim = t.dim()
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return ctypes.byref(d)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check():
    buf = ctypes.create_string_buffer(512)
    code = lib.spd_last_error(buf, 512)
    if code != 0:
        raise SpdError(code, buf.value.decode(errors="replace"))


_PACK = struct.Struct("=Qii4q4q").pack
assert struct.calcsize("=Qii4q4q") == ctypes.sizeof(SpdTensor)
_ZEROS = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())


def _pack(t: Optional[torch.Tensor], name: str, device: int) -> Optional[bytes]:
    """The descriptor of ``t`` as the bytes of an ``spd_tensor``.

    The calls of a serving step pass up to sixteen tensors each and run for a
    few microseconds on the GPU, so what a descriptor costs shows: about 1 us
    like this, 3 us as a ctypes structure that is filled field by field."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s: dtype %s is not supported by libspd" % (name, t.dtype))
    shape = t.shape
    n = len(shape)
    if n > 4:
        raise ValueError("%s has more than 4 dims" % name)
    if t.get_device() != device and t.numel() > 0:
        raise ValueError("%s must be a CUDA tensor on the current device" % name)
    zeros = _ZEROS[n]
    return _PACK(t.data_ptr(), code, n, *shape, *zeros, *t.stride(), *zeros)


def _place(stream):
    """The current device's index and the raw stream of a call."""
    device = torch.cuda.current_device() if torch.cuda.is_available() else -2
    if stream is None:
        return device, (torch._C._cuda_getCurrentRawStream(device) if device >= 0 else None)
    return device, _stream(stream)


def _check_fast():
    if lib.spd_last_error(None, 0) != 0:
        _check()


def _load_marshal():
    """The compiled marshalling of the serving-step calls (csrc/marshal.cpp),
    or None where it was not built: the calls then go through _pack."""
    try:
        from . import _marshal
    except ImportError:
        return None
    _marshal.bind(LIB_PATH, _check)
    return _marshal


_fast = _load_marshal()


def _raw(stream):
    return None if stream is None else _stream(stream)


def msa_block_score(q_idx, k_idx_cache, block_table, seq_lens, req_idx, block_size, scores,
                    idx_scale, stream=None) -> None:
    """Stage 1: fill ``scores`` [Hi, T, NB] with block-max index scores."""
    lib.msa_block_score(_desc(q_idx, "q_idx"), _desc(k_idx_cache, "k_idx_cache"),
                        _desc(block_table, "block_table"), _desc(seq_lens, "seq_lens"),
                        _desc(req_idx, "req_idx"), int(block_size), _desc(scores, "scores"),
                        float(idx_scale), _stream(stream))
    _check()


def msa_select_topk(scores, topk_idx, stream=None) -> None:
    """Stage 2: fill ``topk_idx`` [Hi, T, K] with the top-K block ids per row."""
    lib.msa_select_topk(_desc(scores, "scores"), _desc(topk_idx, "topk_idx"), _stream(stream))
    _check()


def paged_sparse_decode_attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, topk_idx, out,
                                  sm_scale, block_size, k_scale, v_scale, workspace, stream=None) -> None:
    """Stage 3: fill ``out`` [T, Hq, D] (bf16) with attention over the selected blocks.

    ``workspace`` is a CUDA uint8 tensor of at least ``decode_workspace_bytes`` bytes."""
    ws_ptr, ws_bytes = _workspace(workspace)
    lib.paged_sparse_decode_attention(
        _desc(q, "q"), _desc(k_cache, "k_cache"), _desc(v_cache, "v_cache"), _desc(block_table, "block_table"),
        _desc(seq_lens, "seq_lens"), _desc(req_idx, "req_idx"), _desc(topk_idx, "topk_idx"), _desc(out, "out"),
        float(sm_scale), int(block_size), float(k_scale), float(v_scale), ws_ptr, ws_bytes, _stream(stream))
    _check()


def paged_sparse_decode_attention_noalloc(q, k_cache, v_cache, block_table, seq_lens, req_idx, topk_idx, out,
                                          sm_scale, block_size, k_scale, v_scale, stream=None) -> None:
    """Stage 3 for callers that cannot allocate: no workspace argument, the
    library's built-in 16 MiB scratch is used instead (see include/spd.h for
    its limit and its sharing rules)."""
    lib.paged_sparse_decode_attention_noalloc(
        _desc(q, "q"), _desc(k_cache, "k_cache"), _desc(v_cache, "v_cache"), _desc(block_table, "block_table"),
        _desc(seq_lens, "seq_lens"), _desc(req_idx, "req_idx"), _desc(topk_idx, "topk_idx"), _desc(out, "out"),
        float(sm_scale), int(block_size), float(k_scale), float(v_scale), _stream(stream))
    _check()


def paged_decode_attention(q, k_cache, v_cache, block_table, seq_lens, req_idx, out, sm_scale, block_size,
                           k_scale, v_scale, workspace, stream=None) -> None:
    """Dense paged decode: attention over every block of each row."""
    ws_ptr, ws_bytes = _workspace(workspace)
    lib.paged_decode_attention(
        _desc(q, "q"), _desc(k_cache, "k_cache"), _desc(v_cache, "v_cache"), _desc(block_table, "block_table"),
        _desc(seq_lens, "seq_lens"), _desc(req_idx, "req_idx"), _desc(out, "out"), float(sm_scale),
        int(block_size), float(k_scale), float(v_scale), ws_ptr, ws_bytes, _stream(stream))
    _check()


def msa_prefill_block_score(q, index_k_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens,
                            block_size_q, block_size_k, init_blocks, local_blocks, scale, cu_seqblocks_q, out_topk,
                            workspace, stream=None) -> None:
    """Fused prefill score-to-selection: fill ``out_topk`` [Hi, rows, topk]
    with the selected key blocks of every query block of a ragged batch.

    ``workspace`` is a CUDA uint8 tensor of at least
    ``prefill_workspace_bytes(total_q, Hi, NB)`` bytes."""
    ws_ptr, ws_bytes = _workspace(workspace)
    lib.msa_prefill_block_score(
        _desc(q, "q"), _desc(index_k_cache, "index_k_cache"), _desc(block_table, "block_table"),
        _desc(slot_ids, "slot_ids"), _desc(cu_seqlens, "cu_seqlens"), _desc(seq_lens, "seq_lens"),
        _desc(prefix_lens, "prefix_lens"), int(block_size_q), int(block_size_k), int(init_blocks),
        int(local_blocks), float(scale), _desc(cu_seqblocks_q, "cu_seqblocks_q"), _desc(out_topk, "out_topk"),
        ws_ptr, ws_bytes, _stream(stream))
    _check()


def prefill_workspace_bytes(total_q: int, Hi: int, NB: int) -> int:
    """Workspace bytes msa_prefill_block_score needs for these sizes."""
    return int(lib.spd_prefill_workspace_bytes(total_q, Hi, NB))


def paged_assign_slots(new_lens, prefix_lens, slot_ids, free_pages, free_count, n_pages, block_size, block_size_q,
                       block_table, cu_seqlens, cu_seqblocks_q, seq_lens, req_idx, token_lens, slots, free_left,
                       stream=None) -> None:
    """Slots of a serving step: grow ``block_table`` [R, NB] in place from the
    end of ``free_pages`` and fill the offsets, lengths and every token's row,
    length and slot from the requests' ``new_lens`` and ``prefix_lens``."""
    if _fast is not None:
        _fast.paged_assign_slots(new_lens, prefix_lens, slot_ids, free_pages, free_count, n_pages, block_size,
            block_size_q, block_table, cu_seqlens, cu_seqblocks_q, seq_lens, req_idx, token_lens, slots,
            free_left, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_assign_slots(
        _pack(new_lens, "new_lens", d), _pack(prefix_lens, "prefix_lens", d), _pack(slot_ids, "slot_ids", d),
        _pack(free_pages, "free_pages", d), _pack(free_count, "free_count", d), n_pages, block_size, block_size_q,
        _pack(block_table, "block_table", d), _pack(cu_seqlens, "cu_seqlens", d),
        _pack(cu_seqblocks_q, "cu_seqblocks_q", d), _pack(seq_lens, "seq_lens", d), _pack(req_idx, "req_idx", d),
        _pack(token_lens, "token_lens", d), _pack(slots, "slots", d), _pack(free_left, "free_left", d), raw)
    _check_fast()


def paged_norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache, v_cache, eps,
                          interleaved, block_size, k_scale, v_scale, stream=None) -> None:
    """Per-head RMS norm (``q_weight``, ``k_weight`` [D], or None) and rotary
    positions (``cos_sin`` [M, Rd]) of q and k: fill ``q_out`` [T, Hq, D] and
    write k and v into ``slots`` of the caches.  ``v`` and ``v_cache`` may be
    None together (index queries and keys)."""
    if _fast is not None:
        _fast.paged_norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache,
            v_cache, eps, 1 if interleaved else 0, block_size, k_scale, v_scale, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_norm_rope_store(
        _pack(q, "q", d), _pack(k, "k", d), _pack(v, "v", d), _pack(q_weight, "q_weight", d),
        _pack(k_weight, "k_weight", d), _pack(cos_sin, "cos_sin", d), _pack(token_lens, "token_lens", d),
        _pack(slots, "slots", d), _pack(q_out, "q_out", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d),
        eps, 1 if interleaved else 0, block_size, k_scale, v_scale, raw)
    _check_fast()


def paged_prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens, out,
                            sm_scale, block_size, k_scale, v_scale, workspace, stream=None) -> None:
    """Prefill attention: fill ``out`` [total_q, Hq, D] (bf16) with attention
    of a ragged batch of chunks over every key of the paged caches.

    ``workspace`` is a CUDA uint8 tensor of at least
    ``prefill_attention_workspace_bytes`` bytes."""
    if _fast is not None:
        _fast.paged_prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens,
            prefix_lens, out, sm_scale, block_size, k_scale, v_scale, workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_prefill_attention(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d),
        _pack(block_table, "block_table", d), _pack(slot_ids, "slot_ids", d), _pack(cu_seqlens, "cu_seqlens", d),
        _pack(seq_lens, "seq_lens", d), _pack(prefix_lens, "prefix_lens", d), _pack(out, "out", d), sm_scale,
        block_size, k_scale, v_scale, *_scratch(workspace, d), raw)
    _check_fast()


def paged_sparse_prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens, prefix_lens,
                                   topk_idx, block_size_q, cu_seqblocks_q, out, sm_scale, block_size, k_scale,
                                   v_scale, workspace, stream=None) -> None:
    """The same over the key blocks that ``topk_idx`` [Hkv, rows, K] lists for
    each query block of ``block_size_q`` tokens (the rows that
    msa_prefill_block_score writes)."""
    if _fast is not None:
        _fast.paged_sparse_prefill_attention(q, k_cache, v_cache, block_table, slot_ids, cu_seqlens, seq_lens,
            prefix_lens, topk_idx, block_size_q, cu_seqblocks_q, out, sm_scale, block_size, k_scale, v_scale,
            workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_sparse_prefill_attention(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d),
        _pack(block_table, "block_table", d), _pack(slot_ids, "slot_ids", d), _pack(cu_seqlens, "cu_seqlens", d),
        _pack(seq_lens, "seq_lens", d), _pack(prefix_lens, "prefix_lens", d), _pack(topk_idx, "topk_idx", d),
        block_size_q, _pack(cu_seqblocks_q, "cu_seqblocks_q", d), _pack(out, "out", d), sm_scale, block_size, k_scale,
        v_scale, *_scratch(workspace, d), raw)
    _check_fast()


def paged_norm_rope_store_block_scaled(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache, v_cache,
                                       k_scales, v_scales, eps, interleaved, block_size, stream=None) -> None:
    """paged_norm_rope_store into E4M3 caches with one scale for each page and
    kv head: ``k_scales`` and ``v_scales`` [P, Hkv] f32 grow in place, as
    powers of two, with what is stored, and the codes that a page holds
    already follow."""
    if _fast is not None:
        _fast.paged_norm_rope_store_block_scaled(q, k, v, q_weight, k_weight, cos_sin, token_lens, slots, q_out, k_cache,
            v_cache, k_scales, v_scales, eps, 1 if interleaved else 0, block_size, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_norm_rope_store_block_scaled(
        _pack(q, "q", d), _pack(k, "k", d), _pack(v, "v", d), _pack(q_weight, "q_weight", d),
        _pack(k_weight, "k_weight", d), _pack(cos_sin, "cos_sin", d), _pack(token_lens, "token_lens", d),
        _pack(slots, "slots", d), _pack(q_out, "q_out", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d),
        _pack(k_scales, "k_scales", d), _pack(v_scales, "v_scales", d), eps, 1 if interleaved else 0, block_size, raw)
    _check_fast()


def paged_decode_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, req_idx, out,
                                        sm_scale, block_size, workspace, stream=None) -> None:
    """paged_decode_attention over E4M3 caches with one scale for each page and
    kv head (``k_scales``, ``v_scales`` [P, Hkv] f32)."""
    if _fast is not None:
        _fast.paged_decode_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, req_idx,
            out, sm_scale, block_size, workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_decode_attention_block_scaled(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d), _pack(k_scales, "k_scales", d),
        _pack(v_scales, "v_scales", d), _pack(block_table, "block_table", d), _pack(seq_lens, "seq_lens", d),
        _pack(req_idx, "req_idx", d), _pack(out, "out", d), sm_scale, block_size, *_scratch(workspace, d), raw)
    _check_fast()


def paged_sparse_decode_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, req_idx,
                                               topk_idx, out, sm_scale, block_size, workspace, stream=None) -> None:
    """paged_sparse_decode_attention over E4M3 caches with one scale for each
    page and kv head."""
    if _fast is not None:
        _fast.paged_sparse_decode_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens,
            req_idx, topk_idx, out, sm_scale, block_size, workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_sparse_decode_attention_block_scaled(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d), _pack(k_scales, "k_scales", d),
        _pack(v_scales, "v_scales", d), _pack(block_table, "block_table", d), _pack(seq_lens, "seq_lens", d),
        _pack(req_idx, "req_idx", d), _pack(topk_idx, "topk_idx", d), _pack(out, "out", d), sm_scale, block_size,
        *_scratch(workspace, d), raw)
    _check_fast()


def paged_prefill_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, slot_ids, cu_seqlens,
                                         seq_lens, prefix_lens, out, sm_scale, block_size, workspace,
                                         stream=None) -> None:
    """paged_prefill_attention over E4M3 caches with one scale for each page
    and kv head."""
    if _fast is not None:
        _fast.paged_prefill_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, slot_ids,
            cu_seqlens, seq_lens, prefix_lens, out, sm_scale, block_size, workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_prefill_attention_block_scaled(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d), _pack(k_scales, "k_scales", d),
        _pack(v_scales, "v_scales", d), _pack(block_table, "block_table", d), _pack(slot_ids, "slot_ids", d),
        _pack(cu_seqlens, "cu_seqlens", d), _pack(seq_lens, "seq_lens", d), _pack(prefix_lens, "prefix_lens", d),
        _pack(out, "out", d), sm_scale, block_size, *_scratch(workspace, d), raw)
    _check_fast()


def paged_sparse_prefill_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, slot_ids,
                                                cu_seqlens, seq_lens, prefix_lens, topk_idx, block_size_q,
                                                cu_seqblocks_q, out, sm_scale, block_size, workspace,
                                                stream=None) -> None:
    """paged_sparse_prefill_attention over E4M3 caches with one scale for each
    page and kv head."""
    if _fast is not None:
        _fast.paged_sparse_prefill_attention_block_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, slot_ids,
            cu_seqlens, seq_lens, prefix_lens, topk_idx, block_size_q, cu_seqblocks_q, out, sm_scale, block_size,
            workspace, _raw(stream))
        return
    d, raw = _place(stream)
    lib.paged_sparse_prefill_attention_block_scaled(
        _pack(q, "q", d), _pack(k_cache, "k_cache", d), _pack(v_cache, "v_cache", d), _pack(k_scales, "k_scales", d),
        _pack(v_scales, "v_scales", d), _pack(block_table, "block_table", d), _pack(slot_ids, "slot_ids", d),
        _pack(cu_seqlens, "cu_seqlens", d), _pack(seq_lens, "seq_lens", d), _pack(prefix_lens, "prefix_lens", d),
        _pack(topk_idx, "topk_idx", d), block_size_q, _pack(cu_seqblocks_q, "cu_seqblocks_q", d), _pack(out, "out", d),
        sm_scale, block_size, *_scratch(workspace, d), raw)
    _check_fast()


def _scratch(ws, device):
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or ws.get_device() != device:
        raise TypeError("workspace must be a CUDA tensor on the current device")
    if not ws.is_contiguous():  # its bytes are used as one run
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def prefill_attention_workspace_bytes(total_q: int, Hq: int, Hkv: int, D: int, B: int, NB: int, n_rows: int = 0) -> int:
    """Workspace bytes the prefill attention calls need for these capacities
    (``n_rows``: the rows of topk_idx, 0 for paged_prefill_attention)."""
    return int(lib.spd_prefill_attention_workspace_bytes(total_q, Hq, Hkv, D, B, NB, n_rows))


def attention_sdpa(q, k, v, out, sm_scale, causal, stream=None) -> None:
    """Dense GQA attention: fill ``out`` [T, Hq, D] from q [T, Hq, D] and
    k, v [S, Hkv, D]; with ``causal`` query t reads keys j <= t + S - T."""
    lib.attention_sdpa(_desc(q, "q"), _desc(k, "k"), _desc(v, "v"), _desc(out, "out"), float(sm_scale),
                       1 if causal else 0, _stream(stream))
    _check()


def _workspace(ws):
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def set_attention_kernel(policy: int) -> int:
    """0 = tensor-core kernel where it applies (default), 1 = general-layout
    kernel always.  Applies to this thread; returns the previous policy."""
    return int(lib.spd_set_attention_kernel(int(policy)))


STAGE_SCORE, STAGE_SELECT, STAGE_ATTENTION, STAGE_SDPA, STAGE_PREFILL_ATTENTION, STAGE_STORE = 1, 2, 3, 4, 5, 6


def set_kernel_policy(stage: int, policy: int) -> int:
    """Kernel choice of one stage (1 score, 2 select, 3 attention, 4 dense
    attention, 5 prefill attention, 6 norm and store) on this thread: 0 = specialised kernel where it applies
    (default), 1 = general-layout kernel always.  Returns the previous
    policy."""
    old = int(lib.spd_set_kernel_policy(int(stage), int(policy)))
    if old < 0:
        raise ValueError("unknown stage %r" % (stage,))
    return old


def workspace_status(workspace, stream=None) -> int:
    """Status word an attention call left in ``workspace`` (synchronises):
    0 ok, bit 0 a device-side wait timed out.  ``workspace=None`` reads the
    built-in scratch that paged_sparse_decode_attention_noalloc uses on the
    current device."""
    ptr = None if workspace is None else workspace.data_ptr()
    return int(lib.spd_workspace_status(ptr, _stream(stream)))


def launch_count() -> int:
    """Kernels enqueued by libspd in this process so far."""
    return int(lib.spd_launch_count())


def decode_workspace_bytes(T: int, Hq: int, Hkv: int, D: int, NB: int, block_size: int = 128) -> int:
    """Workspace bytes the attention calls need for these capacities."""
    return int(lib.spd_decode_workspace_bytes(T, Hq, Hkv, D, NB, block_size))
