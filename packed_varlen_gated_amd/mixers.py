"""Binding of include/pkv_mixers.h: packed causal softmax attention with grouped
heads, packed linear attention with one decay per head, and the single-token
steps of the recurrences. The same thin marshalling as the package's other
calls: shapes, dtypes and devices are checked, and every step of the
computation runs in the library's HIP kernels on torch's current stream.

* ``attn_varlen(q, k, v, cu_seqlens=None, scale=None, output_lse=True)``
* ``attn_varlen_backward(q, k, v, o, lse, do, cu_seqlens=None, scale=None)``
* ``chunk_linear_attn_varlen(q, k, v, g, cu_seqlens=None, scale=1.0, output_final_state=True)``
* ``chunk_linear_attn_varlen_backward(q, k, v, g, do, cu_seqlens=None, scale=1.0)``
* ``linear_attn_step(q, k, v, g, state, slots=None, scale=1.0)``
* ``kda_step(q, k, v, g, beta, state, slots=None, scale=1.0)``
"""

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import (_check, _dtype_code, _load, _need, _need_shape, _ptr, _stream, _workspace,
               OPT_QK_L2NORM)

FLAG_BAD_SLOT = 16

_NOTHING = contextlib.nullcontext()


def declare(lib):
    """Argument types of the calls (once, when the library is loaded)."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    sizes = [vp, i32, i64, i32, i32, i32, f32, i32]   # cu_seqlens, max_segs, N, three sizes, scale, dtype
    for name, args, res in (
            ("pkv_attn_varlen", [vp] * 3 + sizes + [vp] * 4, i32),
            ("pkv_attn_varlen_backward_workspace_size", [i64, i32, i32, i32, i32, i32], sz),
            ("pkv_attn_varlen_backward", [vp] * 6 + sizes + [vp] * 5 + [sz, vp], i32),
            ("pkv_linear_attn_varlen_workspace_size", [i64, i32, i32, i32, i32, i32], sz),
            ("pkv_linear_attn_varlen", [vp] * 4 + sizes + [vp] * 5 + [sz, vp], i32),
            ("pkv_linear_attn_varlen_backward_workspace_size", [i64, i32, i32, i32, i32, i32], sz),
            ("pkv_linear_attn_varlen_backward", [vp] * 4 + sizes + [vp] * 9 + [sz, vp], i32),
            ("pkv_linear_attn_step", [vp] * 5 + [i64, i32, i32, i32, i32, f32, i32] + [vp] * 4, i32),
            ("pkv_kda_step", [vp] * 6 + [i64, i32, i32, i32, i32, f32, i32, i32] + [vp] * 4, i32)):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res


def _on(device):
    """The call's device as the current one while it launches."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, expected a GPU")
    return _NOTHING if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _slots_of(cu_seqlens, device):
    if cu_seqlens is None:
        return 1
    _need(cu_seqlens, "cu_seqlens", device, torch.int32, 1)
    if cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold max_segs + 1 >= 2 entries")
    return cu_seqlens.shape[0] - 1


def _attn_shapes(q, k, v, cu_seqlens, scale, flags):
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dev, dt, 4)
    B, T, Hq, D = q.shape
    if tuple(k.shape[:2]) != (B, T) or k.shape[3] != D or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [.., N, Hkv, D] with q's N and D")
    Hkv = k.shape[2]
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"q has {Hq} heads, not a multiple of the {Hkv} of k and v")
    segs = _slots_of(cu_seqlens, dev)
    if flags is not None:
        _need(flags, "flags", dev, torch.int32, 1)
        _need_shape(flags, "flags", (1,))
    return dev, code, B * T, Hq, Hkv, D, segs, 1.0 / math.sqrt(D) if scale is None else float(scale)


def attn_varlen(q, k, v, cu_seqlens=None, scale=None, output_lse=True, flags=None, out=None):
    """Packed causal softmax attention.

    q: [1, N, Hq, D] (or [B, T, Hq, D], taken as the flattened [1, B*T, Hq, D]); k, v: the same with
    Hkv heads, a divisor of Hq (query head h reads kv head h // (Hq // Hkv)); cu_seqlens: int32
    [max_segs + 1] or None (one segment); scale: None means 1 / sqrt(D).
    Returns (o like q, lse fp32 [Hq, N] or None). A token attends to itself and the earlier tokens of
    its segment; positions past cu_seqlens[-1] get o = 0, lse = -inf.
    """
    lib = _load()
    dev, code, N, Hq, Hkv, D, segs, scale = _attn_shapes(q, k, v, cu_seqlens, scale, flags)
    o = torch.empty_like(q) if out is None else out
    _need(o, "out", dev, q.dtype, 4)
    _need_shape(o, "out", q.shape)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=dev) if output_lse else None
    with _on(dev):
        _check(lib.pkv_attn_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), segs, N, Hq, Hkv, D, scale, code,
                                   _ptr(o), _ptr(lse), _ptr(flags), _stream(dev)))
    return o, lse


class AttnGrads(NamedTuple):
    dq: torch.Tensor  # like q
    dk: torch.Tensor  # like k
    dv: torch.Tensor  # like v


def attn_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, dtype):
    return int(_load().pkv_attn_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, _dtype_code(dtype)))


def attn_varlen_backward(q, k, v, o, lse, do, cu_seqlens=None, scale=None, flags=None, workspace=None):
    """Reverse pass of ``attn_varlen`` on the same inputs, with the o and lse it returned and
    do = dL/do. Returns AttnGrads; dk and dv are summed over the query heads of their kv head."""
    lib = _load()
    dev, code, N, Hq, Hkv, D, segs, scale = _attn_shapes(q, k, v, cu_seqlens, scale, flags)
    for name, t in (("o", o), ("do", do)):
        _need(t, name, dev, q.dtype, 4)
        _need_shape(t, name, q.shape)
    _need(lse, "lse", dev, torch.float32, 2)
    _need_shape(lse, "lse", (Hq, N))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = int(lib.pkv_attn_varlen_backward_workspace_size(N, Hq, Hkv, D, segs, code))
    workspace, ws_bytes = _workspace(workspace, need, dev)
    with _on(dev):
        _check(lib.pkv_attn_varlen_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                            _ptr(cu_seqlens), segs, N, Hq, Hkv, D, scale, code, _ptr(dq), _ptr(dk),
                                            _ptr(dv), _ptr(flags), _ptr(workspace), ws_bytes, _stream(dev)))
    return AttnGrads(dq, dk, dv)


def _linear_shapes(q, k, v, g, cu_seqlens, states, flags):
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dev, dt, 4)
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    if tuple(k.shape) != tuple(q.shape):
        raise ValueError("q and k must have the same shape")
    if tuple(v.shape[:3]) != (B, T, H):
        raise ValueError("v must be [.., N, H, Dv]")
    _need(g, "g", dev, torch.float32, 1)
    _need_shape(g, "g", (H,))
    segs = _slots_of(cu_seqlens, dev)
    for name, t in states:
        if t is not None:
            _need(t, name, dev, torch.float32, 4)
            _need_shape(t, name, (segs, H, Dk, Dv))
    if flags is not None:
        _need(flags, "flags", dev, torch.int32, 1)
        _need_shape(flags, "flags", (1,))
    return dev, code, B * T, H, Dk, Dv, segs


def chunk_linear_attn_varlen_workspace_size(N, H, Dk, Dv, max_segs, dtype):
    return int(_load().pkv_linear_attn_varlen_workspace_size(N, H, Dk, Dv, max_segs, _dtype_code(dtype)))


def chunk_linear_attn_varlen(q, k, v, g, cu_seqlens=None, scale=1.0, output_final_state=True, flags=None, out=None,
                             workspace=None, initial_state=None):
    """Packed linear attention with one decay per head: S_t = exp(g[h]) S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t, S reset (or set to the slot's initial state) at every segment start.

    q, k: [1, N, H, Dk] (or [B, T, H, Dk], flattened); v: [.., H, Dv]; g: fp32 [H] log decays (a
    constant of the layer); cu_seqlens: int32 [max_segs + 1] or None (one segment); initial_state:
    fp32 [max_segs, H, Dk, Dv] or None.
    Returns (o like v, final_state fp32 [max_segs, H, Dk, Dv] or None).
    """
    lib = _load()
    dev, code, N, H, Dk, Dv, segs = _linear_shapes(q, k, v, g, cu_seqlens, [("initial_state", initial_state)], flags)
    o = torch.empty_like(v) if out is None else out
    _need(o, "out", dev, v.dtype, 4)
    _need_shape(o, "out", v.shape)
    fs = torch.empty(segs, H, Dk, Dv, dtype=torch.float32, device=dev) if output_final_state else None
    need = int(lib.pkv_linear_attn_varlen_workspace_size(N, H, Dk, Dv, segs, code))
    workspace, ws_bytes = _workspace(workspace, need, dev)
    with _on(dev):
        _check(lib.pkv_linear_attn_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu_seqlens), segs, N, H, Dk, Dv,
                                          float(scale), code, _ptr(initial_state), _ptr(o), _ptr(fs), _ptr(flags),
                                          _ptr(workspace), ws_bytes, _stream(dev)))
    return o, fs


class LinearAttnGrads(NamedTuple):
    dq: torch.Tensor                         # like q
    dk: torch.Tensor                         # like k
    dv: torch.Tensor                         # like v
    d_initial_state: Optional[torch.Tensor]  # fp32 [max_segs, H, Dk, Dv] or None


def chunk_linear_attn_varlen_backward_workspace_size(N, H, Dk, Dv, max_segs, dtype):
    return int(_load().pkv_linear_attn_varlen_backward_workspace_size(N, H, Dk, Dv, max_segs, _dtype_code(dtype)))


def chunk_linear_attn_varlen_backward(q, k, v, g, do, cu_seqlens=None, scale=1.0, initial_state=None,
                                      dfinal_state=None, output_d_initial_state=None, flags=None, workspace=None):
    """Reverse pass of ``chunk_linear_attn_varlen`` on the same inputs.

    do: dL/do; dfinal_state: fp32 [max_segs, H, Dk, Dv] or None (dL/dfinal_state). Returns
    LinearAttnGrads; d_initial_state is returned when ``output_d_initial_state`` is true (default:
    when initial_state is given). The decays are constants: they get no gradient.
    """
    lib = _load()
    dev, code, N, H, Dk, Dv, segs = _linear_shapes(
        q, k, v, g, cu_seqlens, [("initial_state", initial_state), ("dfinal_state", dfinal_state)], flags)
    _need(do, "do", dev, v.dtype, 4)
    _need_shape(do, "do", v.shape)
    if output_d_initial_state is None:
        output_d_initial_state = initial_state is not None
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dinit = torch.empty(segs, H, Dk, Dv, dtype=torch.float32, device=dev) if output_d_initial_state else None
    need = int(lib.pkv_linear_attn_varlen_backward_workspace_size(N, H, Dk, Dv, segs, code))
    workspace, ws_bytes = _workspace(workspace, need, dev)
    with _on(dev):
        _check(lib.pkv_linear_attn_varlen_backward(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu_seqlens), segs, N, H, Dk, Dv, float(scale), code,
            _ptr(initial_state), _ptr(do), _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dinit),
            _ptr(flags), _ptr(workspace), ws_bytes, _stream(dev)))
    return LinearAttnGrads(dq, dk, dv, dinit)


def _step_shapes(q, k, v, state, slots, out, flags):
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dev, dt, 3)
    R, H, Dk = q.shape
    Dv = v.shape[2]
    if tuple(k.shape) != tuple(q.shape):
        raise ValueError("q and k must have the same shape")
    if tuple(v.shape[:2]) != (R, H):
        raise ValueError("v must be [R, H, Dv]")
    _need(state, "state", dev, torch.float32, 4)
    S = state.shape[0]
    _need_shape(state, "state", (S, H, Dk, Dv))
    if slots is not None:
        _need(slots, "slots", dev, torch.int32, 1)
        _need_shape(slots, "slots", (R,))
    elif R > S:
        raise ValueError(f"{R} rows for {S} state slots")
    o = torch.empty_like(v) if out is None else out
    _need(o, "out", dev, dt, 3)
    _need_shape(o, "out", v.shape)
    if flags is not None:
        _need(flags, "flags", dev, torch.int32, 1)
        _need_shape(flags, "flags", (1,))
    return dev, code, R, S, H, Dk, Dv, o


def linear_attn_step(q, k, v, g, state, slots=None, scale=1.0, out=None, flags=None):
    """One token of each of R requests through the recurrence of ``chunk_linear_attn_varlen``.

    q, k: [R, H, Dk]; v: [R, H, Dv]; g: fp32 [H]; state: fp32 [S, H, Dk, Dv], updated in place (the
    final states of the packed call are such states); slots: int32 [R], request r's state slot, or
    None (slot r). Returns o [R, H, Dv]. A negative slot is an idle row (o = 0, no state touched); a
    slot past the last one, or named by an earlier row too, is treated the same and sets
    ``FLAG_BAD_SLOT`` in flags.
    """
    lib = _load()
    dev, code, R, S, H, Dk, Dv, o = _step_shapes(q, k, v, state, slots, out, flags)
    _need(g, "g", dev, torch.float32, 1)
    _need_shape(g, "g", (H,))
    with _on(dev):
        _check(lib.pkv_linear_attn_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(slots), R, S, H, Dk, Dv,
                                        float(scale), code, _ptr(state), _ptr(o), _ptr(flags), _stream(dev)))
    return o


def kda_step(q, k, v, g, beta, state, slots=None, scale=1.0, out=None, flags=None, use_qk_l2norm_in_kernel=False):
    """One token of each of R requests through the recurrence of ``chunk_kda_varlen``
    (S = diag(exp g) S + beta k v^T, o = scale S^T q).

    q, k, g: [R, H, Dk]; v: [R, H, Dv]; beta: [R, H]; state and slots as for ``linear_attn_step``.
    """
    lib = _load()
    dev, code, R, S, H, Dk, Dv, o = _step_shapes(q, k, v, state, slots, out, flags)
    _need(g, "g", dev, q.dtype, 3)
    _need_shape(g, "g", q.shape)
    _need(beta, "beta", dev, q.dtype, 2)
    _need_shape(beta, "beta", (R, H))
    with _on(dev):
        _check(lib.pkv_kda_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(slots), R, S, H, Dk, Dv,
                                float(scale), code, OPT_QK_L2NORM if use_qk_l2norm_in_kernel else 0, _ptr(state),
                                _ptr(o), _ptr(flags), _stream(dev)))
    return o
