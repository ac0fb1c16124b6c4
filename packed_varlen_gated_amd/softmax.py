"""Binding of include/pkv_softmax.h: what stands around ``attn_varlen`` in a softmax
layer, for training and for serving. The same thin marshalling as the package's other
calls: shapes, dtypes and devices are checked, and every step of the computation runs
in the library's HIP kernels on torch's current stream.

* ``qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)``
* ``qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq)``
* ``attn_window_varlen(q, k, v, window, sinks=0, cu_seqlens=None, scale=None, output_lse=True)``
* ``attn_window_varlen_backward(q, k, v, o, lse, do, window, sinks=0, cu_seqlens=None, scale=None)``
* ``paged_kv_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None)``
* ``attn_paged(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, window=None, sinks=0, scale=None)``
"""

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import PKV_BF16
from .mixers import (AttnGrads, _attn_shapes, _code, _dtype_code, _flags_of, _load, _need, _need_shape, _ptr, _run,
                     _scratch, _shape, _tensors)

FLAG_BAD_PAGE = 32
FLAG_BAD_LENGTH = 64
OPT_ROPE_INTERLEAVED = 2


def declare(lib):
    """Argument types of the calls (once, when the library is loaded)."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    rope = [vp] * 4 + [i64, i32, i32, i32, i32, f32, i32, i32]   # weights, positions, inv_freq, sizes, eps, ..
    attn = [vp, i32, i64, i32, i32, i32, f32, i32, i32, i32]     # cu_seqlens, sizes, scale, dtype, window, sinks
    pages = [vp, vp, vp, i64] + [i32] * 3                        # table, lengths, cu_seqlens, N, R, ..
    for name, args, res in (
            ("pkv_qk_norm_rope", [vp, vp, i64, i64] + rope + [vp] * 3, i32),
            ("pkv_qk_norm_rope_backward_workspace_size", [i64, i32, i32, i32, i32], sz),
            ("pkv_qk_norm_rope_backward", [vp, vp, i64, i64, vp, vp] + rope + [vp] * 5 + [sz, vp], i32),
            ("pkv_attn_window_varlen", [vp] * 3 + attn + [vp] * 4, i32),
            ("pkv_attn_window_varlen_backward_workspace_size", [i64] + [i32] * 7, sz),
            ("pkv_attn_window_varlen_backward", [vp] * 6 + attn + [vp] * 5 + [sz, vp], i32),
            ("pkv_paged_kv_append", [vp, vp, i64, i64] + pages + [i32] * 4 + [vp] * 4, i32),
            ("pkv_attn_paged_workspace_size", [i64] + [i32] * 5, sz),
            ("pkv_attn_paged", [vp] * 3 + pages + [i32] * 4 + [f32, i32, i32, i32] + [vp] * 4 + [sz, vp], i32)):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res


def _heads(t, name, device, dtype, shape):
    """Tokens of dense heads [.., H, D], any distance apart: the distance in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected device {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dims, got shape {tuple(t.shape)}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[-2] * shape[-1]
    st = t.stride()
    if st[-1] != 1 or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if len(shape) == 4 and shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError(f"{name}: the tokens must be equally far apart")
    return st[-3] if shape[-3] > 1 or len(shape) == 3 or shape[0] == 1 else st[0]


def _rope_shapes(q, k, q_weight, k_weight, positions, inv_freq, interleaved):
    dev, dt = q.get_device(), q.dtype
    code = _code(dt)
    if q.dim() != 4:
        raise ValueError(f"q must have 4 dims, got shape {tuple(q.shape)}")
    B, T, Hq, D = q.shape
    qs = _heads(q, "q", dev, dt, q.shape)
    ks = _heads(k, "k", dev, dt, (B, T, k.shape[2] if k.dim() == 4 else 1, D))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _tensors(dev, torch.float32, 1, **{name: w})
            _shape(w, name, (D,))
    if positions is not None:
        _need(positions, "positions", q.device, torch.int32)
        if positions.numel() != B * T:
            raise ValueError(f"positions must hold {B * T} entries, got shape {tuple(positions.shape)}")
    rot = 0
    if inv_freq is not None:
        _tensors(dev, torch.float32, 1, inv_freq=inv_freq)
        rot = 2 * inv_freq.shape[0]
        if rot > D or rot % 16 != 0:
            raise ValueError(f"inv_freq must hold rot_dim / 2 entries, rot_dim a multiple of 16 up to {D}")
    # (one token has no distance to the next: any will do)
    Hkv = k.shape[2]
    if B * T == 1:
        qs, ks = Hq * D, Hkv * D
    return dev, code, B * T, Hq, Hkv, D, rot, qs, ks, OPT_ROPE_INTERLEAVED if interleaved else 0


def qk_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps=1e-6, interleaved=False,
                 out=None):
    """RMS norm of every head of q and k and the rotation by position, in one pass.

    q: [1, N, Hq, D] (or [B, T, Hq, D], taken as the flattened [1, B*T, Hq, D]); k: the same with Hkv
    heads; both may be views of one projection's result (dense heads, tokens equally far apart).
    q_weight, k_weight: fp32 [D] or None (1). positions: int32, N entries of any shape (those of
    ``eod_to_segment_ids``), or None (0 .. N - 1); a negative one marks a row to leave out, whose
    results are 0. inv_freq: fp32 [rot_dim / 2], the angle per position of every pair of the first
    rot_dim channels, or None (no rotation); pair i is channels i and i + rot_dim / 2, or with
    ``interleaved`` 2 i and 2 i + 1. out: (q_out, k_out) or None.
    Returns (q_out, k_out), contiguous.
    """
    lib = _load()
    dev, code, N, Hq, Hkv, D, rot, qs, ks, opt = _rope_shapes(q, k, q_weight, k_weight, positions, inv_freq,
                                                              interleaved)
    if out is None:
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    else:
        qo, ko = out
        _tensors(dev, q.dtype, 4, q_out=qo, k_out=ko)
        _shape(qo, "q_out", q.shape)
        _shape(ko, "k_out", k.shape)
    _run(lib.pkv_qk_norm_rope, dev, q.data_ptr(), k.data_ptr(), qs, ks, _ptr(q_weight), _ptr(k_weight), _ptr(positions),
         _ptr(inv_freq), N, Hq, Hkv, D, rot, float(eps), code, opt, qo.data_ptr(), ko.data_ptr())
    return qo, ko


class QkNormRopeGrads(NamedTuple):
    dq: torch.Tensor                   # like q, contiguous
    dk: torch.Tensor                   # like k, contiguous
    dq_weight: Optional[torch.Tensor]  # fp32 [D], or None without q_weight
    dk_weight: Optional[torch.Tensor]


def qk_norm_rope_backward_workspace_size(N, Hq, Hkv, D, dtype):
    return int(_load().pkv_qk_norm_rope_backward_workspace_size(N, Hq, Hkv, D, _dtype_code(dtype)))


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps=1e-6,
                          interleaved=False, workspace=None):
    """Reverse pass of ``qk_norm_rope`` on the same inputs, with the gradients of its results.
    Returns QkNormRopeGrads; a weight that is None has no gradient."""
    lib = _load()
    dev, code, N, Hq, Hkv, D, rot, qs, ks, opt = _rope_shapes(q, k, q_weight, k_weight, positions, inv_freq,
                                                              interleaved)
    _tensors(dev, q.dtype, 4, dq_out=dq_out, dk_out=dk_out)
    _shape(dq_out, "dq_out", q.shape)
    _shape(dk_out, "dk_out", k.shape)
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    ws_bytes = 0
    if dwq is not None or dwk is not None:
        workspace, ws_bytes = _scratch(workspace, lib.pkv_qk_norm_rope_backward_workspace_size(N, Hq, Hkv, D, code), q)
    _run(lib.pkv_qk_norm_rope_backward, dev, q.data_ptr(), k.data_ptr(), qs, ks, dq_out.data_ptr(), dk_out.data_ptr(),
         _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq), N, Hq, Hkv, D, rot, float(eps), code, opt,
         dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk), _ptr(workspace), ws_bytes)
    return QkNormRopeGrads(dq, dk, dwq, dwk)


def attn_window_varlen(q, k, v, window, sinks=0, cu_seqlens=None, scale=None, output_lse=True, flags=None, out=None):
    """``attn_varlen`` through a sliding window: a token attends to itself, the window - 1 tokens
    before it and the first ``sinks`` (at most 64) tokens of its segment.

    Arguments and results otherwise as for ``attn_varlen``.
    """
    lib = _load()
    dev, code, N, Hq, Hkv, D, segs, scale = _attn_shapes(q, k, v, cu_seqlens, scale, flags)
    if out is None:
        out = torch.empty_like(q)
    else:
        _tensors(dev, q.dtype, 4, out=out)
        _shape(out, "out", q.shape)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=q.device) if output_lse else None
    _run(lib.pkv_attn_window_varlen, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(cu_seqlens), segs, N, Hq, Hkv,
         D, scale, code, _int32(window, "window"), _int32(sinks, "sinks"), out.data_ptr(), _ptr(lse), _ptr(flags))
    return out, lse


def _int32(x, name):
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name} is out of range: {x}")
    return int(x)


def attn_window_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, dtype, window, sinks=0):
    return int(_load().pkv_attn_window_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, _dtype_code(dtype),
                                                                      window, sinks))


def attn_window_varlen_backward(q, k, v, o, lse, do, window, sinks=0, cu_seqlens=None, scale=None, flags=None,
                                workspace=None):
    """Reverse pass of ``attn_window_varlen`` on the same inputs, with the o and lse it returned and
    do = dL/do. Returns AttnGrads; dk and dv are summed over the query heads of their kv head."""
    lib = _load()
    dev, code, N, Hq, Hkv, D, segs, scale = _attn_shapes(q, k, v, cu_seqlens, scale, flags)
    _tensors(dev, q.dtype, 4, o=o, do=do)
    _shape(o, "o", q.shape)
    _shape(do, "do", q.shape)
    _tensors(dev, torch.float32, 2, lse=lse)
    _shape(lse, "lse", (Hq, N))
    window, sinks = _int32(window, "window"), _int32(sinks, "sinks")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    workspace, ws_bytes = _scratch(workspace, lib.pkv_attn_window_varlen_backward_workspace_size(
        N, Hq, Hkv, D, segs, code, window, sinks), q)
    _run(lib.pkv_attn_window_varlen_backward, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
         lse.data_ptr(), do.data_ptr(), _ptr(cu_seqlens), segs, N, Hq, Hkv, D, scale, code, window, sinks,
         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(flags), _ptr(workspace), ws_bytes)
    return AttnGrads(dq, dk, dv)


def _paged_shapes(N, Hkv, D, k_pages, v_pages, page_table, kv_lens, cu_seqlens, flags, dev, dt):
    _tensors(dev, dt, 4, k_pages=k_pages, v_pages=v_pages)
    pages, size, ph, pd = k_pages.shape
    if ph != Hkv or pd != D or v_pages.shape != k_pages.shape:
        raise ValueError(f"k_pages and v_pages must both be [pages, page_size, {Hkv}, {D}]")
    _tensors(dev, torch.int32, 2, page_table=page_table)
    _tensors(dev, torch.int32, 1, kv_lens=kv_lens)
    R, width = page_table.shape
    _shape(kv_lens, "kv_lens", (R,))
    if cu_seqlens is not None:
        _tensors(dev, torch.int32, 1, cu_seqlens=cu_seqlens)
        _shape(cu_seqlens, "cu_seqlens", (R + 1,))
    elif N != R:
        raise ValueError(f"{N} new tokens for {R} requests need cu_seqlens")
    _flags_of(flags, dev)
    return R, size, pages, width


def paged_kv_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, flags=None):
    """New tokens' keys and values into a paged cache (in place).

    k, v: [N, Hkv, D] (dense heads, tokens equally far apart); k_pages, v_pages: [pages, page_size,
    Hkv, D], page_size a multiple of 16; page_table: int32 [R, max_pages], request r's place i lies in
    page page_table[r, i // page_size]; kv_lens: int32 [R], the requests' tokens with the new ones;
    cu_seqlens: int32 [R + 1], request r's new tokens are [cu[r], cu[r + 1]) and its last ones, or None
    (one each, N = R). A request with kv_lens 0 is idle. A length that its row of the table cannot hold
    sets ``FLAG_BAD_LENGTH`` in flags, a page that does not exist ``FLAG_BAD_PAGE``; such tokens are left out.
    """
    lib = _load()
    dev, dt = k.get_device(), k.dtype
    code = _code(dt)
    if k.dim() != 3:
        raise ValueError(f"k must have 3 dims, got shape {tuple(k.shape)}")
    N, Hkv, D = k.shape
    ks, vs = _heads(k, "k", dev, dt, k.shape), _heads(v, "v", dev, dt, k.shape)
    if N == 1:
        ks = vs = Hkv * D
    R, size, pages, width = _paged_shapes(N, Hkv, D, k_pages, v_pages, page_table, kv_lens, cu_seqlens, flags, dev, dt)
    _run(lib.pkv_paged_kv_append, dev, k.data_ptr(), v.data_ptr(), ks, vs, page_table.data_ptr(), kv_lens.data_ptr(),
         _ptr(cu_seqlens), N, R, Hkv, D, size, pages, width, code, k_pages.data_ptr(), v_pages.data_ptr(), _ptr(flags))


def attn_paged_workspace_size(N, R, Hq, Hkv, D, dtype, chunks=True):
    """chunks: whether the call has cu_seqlens (without it bf16 calls at D 64 and 128 need a fifth)."""
    return int(_paged_workspace_size(_load(), N, R, Hq, Hkv, D, _dtype_code(dtype), chunks))


def _paged_workspace_size(lib, N, R, Hq, Hkv, D, code, chunks):
    if not chunks and code == PKV_BF16 and D > 32:
        N = R = 1
    return lib.pkv_attn_paged_workspace_size(N, R, Hq, Hkv, D, code)


def attn_paged(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, window=None, sinks=0, scale=None,
               output_lse=False, flags=None, out=None, workspace=None):
    """Softmax attention of new tokens over a paged cache that already holds their keys and values.

    q: [N, Hq, D], Hq a multiple of the cache's heads; the cache, page_table, kv_lens, cu_seqlens and
    flags as for ``paged_kv_append``: with cu_seqlens chunks of new tokens, without it one token of
    each request. window, sinks: as for ``attn_window_varlen``, or None (no window); scale: None means
    1 / sqrt(D).
    Returns (o like q, lse fp32 [Hq, N] or None). An idle request's rows and those past
    cu_seqlens[-1] get o = 0, lse = -inf.
    """
    lib = _load()
    dev, dt = q.get_device(), q.dtype
    code = _code(dt)
    _tensors(dev, dt, 3, q=q)
    N, Hq, D = q.shape
    if k_pages.dim() != 4 or k_pages.shape[2] < 1 or Hq % k_pages.shape[2] != 0:
        raise ValueError(f"k_pages must be [pages, page_size, Hkv, D] with Hkv a divisor of q's {Hq} heads")
    Hkv = k_pages.shape[2]
    R, size, pages, width = _paged_shapes(N, Hkv, D, k_pages, v_pages, page_table, kv_lens, cu_seqlens, flags, dev, dt)
    if window is None:
        window, sinks = 0, 0
    elif window < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _tensors(dev, dt, 3, out=out)
        _shape(out, "out", q.shape)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=q.device) if output_lse else None
    workspace, ws_bytes = _scratch(
        workspace, _paged_workspace_size(lib, N, R, Hq, Hkv, D, code, cu_seqlens is not None), q)
    _run(lib.pkv_attn_paged, dev, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
         kv_lens.data_ptr(), _ptr(cu_seqlens), N, R, Hq, Hkv, D, size, pages, width,
         1.0 / math.sqrt(D) if scale is None else float(scale), code, _int32(window, "window"), _int32(sinks, "sinks"),
         out.data_ptr(), _ptr(lse), _ptr(flags), _ptr(workspace), ws_bytes)
    return out, lse
