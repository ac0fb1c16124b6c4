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

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _check, _dtype_code, _load, _need, _need_shape, _workspace, OPT_QK_L2NORM, PKV_BF16

FLAG_BAD_SLOT = 16

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


# A decoding step's kernel takes a few microseconds, so the checks of a call that
# passes them are kept short: _fit asks everything of several tensors at once, and
# only where it says no does _need find out what is wrong.
def _fit(index, dtype, ndim, *tensors):
    try:
        for t in tensors:
            if t.get_device() != index or t.dtype is not dtype or t.dim() != ndim or not t.is_contiguous():
                return False
        return True
    except AttributeError:
        return False


def _tensors(device, dtype, ndim, **tensors):
    if not _fit(device, dtype, ndim, *tensors.values()):
        dev = next((t.device for t in tensors.values() if isinstance(t, torch.Tensor) and t.get_device() == device),
                   torch.device("cuda", device) if device >= 0 else torch.device("cpu"))
        for name, t in tensors.items():
            _need(t, name, dev, dtype, ndim)


def _shape(t, name, shape):
    if t.shape != shape:
        _need_shape(t, name, shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run(fn, device, *args):
    """The call on the device's current stream, with the device as the current one."""
    if device < 0:
        raise ValueError("the tensors are on the CPU, expected a GPU")
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != 0:
        _check(status)


def _code(dtype):
    return PKV_BF16 if dtype is torch.bfloat16 else _dtype_code(dtype)


def _flags_of(flags, device):
    if flags is not None:
        _tensors(device, torch.int32, 1, flags=flags)
        _shape(flags, "flags", (1,))


def _slots_of(cu_seqlens, device):
    if cu_seqlens is None:
        return 1
    _tensors(device, torch.int32, 1, cu_seqlens=cu_seqlens)
    if cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold max_segs + 1 >= 2 entries")
    return cu_seqlens.shape[0] - 1


def _scratch(workspace, need, q):
    if need <= 0:
        return None, 0
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=q.device), need
    return _workspace(workspace, need, q.device)


def _attn_shapes(q, k, v, cu_seqlens, scale, flags):
    dev, dt = q.get_device(), q.dtype
    code = _code(dt)
    _tensors(dev, dt, 4, q=q, k=k, v=v)
    B, T, Hq, D = q.shape
    kb, kt, Hkv, kd = k.shape
    if kb != B or kt != T or kd != D or v.shape != k.shape:
        raise ValueError("k and v must be [.., N, Hkv, D] with q's N and D")
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"q has {Hq} heads, not a multiple of the {Hkv} of k and v")
    segs = _slots_of(cu_seqlens, dev)
    _flags_of(flags, dev)
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
    if out is None:
        out = torch.empty_like(q)
    else:
        _tensors(dev, q.dtype, 4, out=out)
        _shape(out, "out", q.shape)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=q.device) if output_lse else None
    _run(lib.pkv_attn_varlen, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(cu_seqlens), segs, N, Hq, Hkv, D,
         scale, code, out.data_ptr(), _ptr(lse), _ptr(flags))
    return out, lse


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
    _tensors(dev, q.dtype, 4, o=o, do=do)
    _shape(o, "o", q.shape)
    _shape(do, "do", q.shape)
    _tensors(dev, torch.float32, 2, lse=lse)
    _shape(lse, "lse", (Hq, N))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    workspace, ws_bytes = _scratch(workspace, lib.pkv_attn_varlen_backward_workspace_size(N, Hq, Hkv, D, segs, code), q)
    _run(lib.pkv_attn_varlen_backward, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
         do.data_ptr(), _ptr(cu_seqlens), segs, N, Hq, Hkv, D, scale, code, dq.data_ptr(), dk.data_ptr(),
         dv.data_ptr(), _ptr(flags), _ptr(workspace), ws_bytes)
    return AttnGrads(dq, dk, dv)


def _linear_shapes(q, k, v, g, cu_seqlens, states, flags):
    dev, dt = q.get_device(), q.dtype
    code = _code(dt)
    _tensors(dev, dt, 4, q=q, k=k, v=v)
    B, T, H, Dk = q.shape
    vb, vt, vh, Dv = v.shape
    if k.shape != q.shape:
        raise ValueError("q and k must have the same shape")
    if vb != B or vt != T or vh != H:
        raise ValueError("v must be [.., N, H, Dv]")
    _tensors(dev, torch.float32, 1, g=g)
    _shape(g, "g", (H,))
    segs = _slots_of(cu_seqlens, dev)
    for name, t in states.items():
        if t is not None:
            _tensors(dev, torch.float32, 4, **{name: t})
            _shape(t, name, (segs, H, Dk, Dv))
    _flags_of(flags, dev)
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
    dev, code, N, H, Dk, Dv, segs = _linear_shapes(q, k, v, g, cu_seqlens, dict(initial_state=initial_state), flags)
    if out is None:
        out = torch.empty_like(v)
    else:
        _tensors(dev, v.dtype, 4, out=out)
        _shape(out, "out", v.shape)
    fs = torch.empty(segs, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
    workspace, ws_bytes = _scratch(workspace, lib.pkv_linear_attn_varlen_workspace_size(N, H, Dk, Dv, segs, code), q)
    _run(lib.pkv_linear_attn_varlen, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(cu_seqlens),
         segs, N, H, Dk, Dv, float(scale), code, _ptr(initial_state), out.data_ptr(), _ptr(fs), _ptr(flags),
         _ptr(workspace), ws_bytes)
    return out, fs


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
        q, k, v, g, cu_seqlens, dict(initial_state=initial_state, dfinal_state=dfinal_state), flags)
    _tensors(dev, v.dtype, 4, do=do)
    _shape(do, "do", v.shape)
    if output_d_initial_state is None:
        output_d_initial_state = initial_state is not None
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dinit = torch.empty(segs, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_d_initial_state else None
    workspace, ws_bytes = _scratch(
        workspace, lib.pkv_linear_attn_varlen_backward_workspace_size(N, H, Dk, Dv, segs, code), q)
    _run(lib.pkv_linear_attn_varlen_backward, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
         _ptr(cu_seqlens), segs, N, H, Dk, Dv, float(scale), code, _ptr(initial_state), do.data_ptr(),
         _ptr(dfinal_state), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dinit), _ptr(flags), _ptr(workspace),
         ws_bytes)
    return LinearAttnGrads(dq, dk, dv, dinit)


def _step_shapes(q, k, v, state, slots, out, flags):
    dev, dt = q.get_device(), q.dtype
    code = _code(dt)
    _tensors(dev, dt, 3, q=q, k=k, v=v)
    R, H, Dk = q.shape
    vr, vh, Dv = v.shape
    if k.shape != q.shape:
        raise ValueError("q and k must have the same shape")
    if vr != R or vh != H:
        raise ValueError("v must be [R, H, Dv]")
    _tensors(dev, torch.float32, 4, state=state)
    S, sh, sk, sv = state.shape
    if sh != H or sk != Dk or sv != Dv:
        _need_shape(state, "state", (S, H, Dk, Dv))
    if slots is not None:
        _tensors(dev, torch.int32, 1, slots=slots)
        if slots.shape[0] != R:
            _need_shape(slots, "slots", (R,))
    elif R > S:
        raise ValueError(f"{R} rows for {S} state slots")
    if out is None:
        out = torch.empty_like(v)
    else:
        _tensors(dev, dt, 3, out=out)
        _shape(out, "out", v.shape)
    _flags_of(flags, dev)
    return dev, code, R, S, H, Dk, Dv, out


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
    _tensors(dev, torch.float32, 1, g=g)
    if g.shape[0] != H:
        _need_shape(g, "g", (H,))
    _run(lib.pkv_linear_attn_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(slots), R, S, H,
         Dk, Dv, float(scale), code, state.data_ptr(), o.data_ptr(), _ptr(flags))
    return o


def kda_step(q, k, v, g, beta, state, slots=None, scale=1.0, out=None, flags=None, use_qk_l2norm_in_kernel=False):
    """One token of each of R requests through the recurrence of ``chunk_kda_varlen``
    (S = diag(exp g) S + beta k v^T, o = scale S^T q).

    q, k, g: [R, H, Dk]; v: [R, H, Dv]; beta: [R, H]; state and slots as for ``linear_attn_step``.
    """
    lib = _load()
    dev, code, R, S, H, Dk, Dv, o = _step_shapes(q, k, v, state, slots, out, flags)
    _tensors(dev, q.dtype, 3, g=g)
    _shape(g, "g", q.shape)
    _tensors(dev, q.dtype, 2, beta=beta)
    _shape(beta, "beta", (R, H))
    _run(lib.pkv_kda_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(slots),
         R, S, H, Dk, Dv, float(scale), code, OPT_QK_L2NORM if use_qk_l2norm_in_kernel else 0, state.data_ptr(),
         o.data_ptr(), _ptr(flags))
    return o
