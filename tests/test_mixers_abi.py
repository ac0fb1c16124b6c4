"""include/pkv_mixers.h without a GPU: every declared function is exported, and
bad arguments are refused, by the library and by the binding, before anything
is launched."""

import ctypes
import os
import re

import pytest
import torch

import packed_varlen_gated_amd as pkv
from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(pkv.LIB_PATH):
        from packed_varlen_gated_amd import build
        build.build(verbose=False)
    return pkv.library()


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pkv_mixers.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pkv_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 9, names
    for n in names:
        assert hasattr(lib, n), n


def A(i, off=0):
    """A fake device address, never dereferenced."""
    return ctypes.c_void_p((i << 32) + off)


P, NUL = ctypes.c_void_p(0x1000), None
BIG = 1 << 30


def _call(fn, base, kw):
    assert set(kw) <= set(base)
    return fn(*{**base, **kw}.values())


ATTN = dict(q=A(1), k=A(2), v=A(3), cu=P, max_segs=4, N=256, Hq=4, Hkv=2, D=64, scale=1.0, dtype=0, o=A(4), lse=A(5),
            flags=NUL, stream=NUL)
ATTN_BAD = [
    (dict(q=NUL), 1), (dict(k=NUL), 1), (dict(v=NUL), 1), (dict(o=NUL), 1), (dict(N=0), 1), (dict(N=1 << 31), 1),
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(Hq=1 << 17), 1), (dict(max_segs=0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(D=48), 2), (dict(D=256), 2),
    (dict(dtype=2), 2), (dict(N=(1 << 31) - 1, Hq=64, Hkv=64), 1),
    (dict(max_segs=1 << 21), 1), (dict(q=A(1, 2)), 1), (dict(k=A(2, 8)), 1),
]


@pytest.mark.parametrize("kw,code", ATTN_BAD + [
    (dict(o=A(1, 64)), 1), (dict(o=A(3)), 1), (dict(o=A(4, 4)), 1), (dict(lse=A(5, 2)), 1), (dict(lse=A(4, 64)), 1),
    (dict(flags=A(4)), 1)])
def test_attn_refusals(lib, kw, code):
    assert _call(lib.pkv_attn_varlen, ATTN, kw) == code


ATTN_BWD = dict(q=A(1), k=A(2), v=A(3), o=A(4), lse=A(5), do=A(6), cu=P, max_segs=4, N=256, Hq=4, Hkv=2, D=64,
                scale=1.0, dtype=0, dq=A(7), dk=A(8), dv=A(9), flags=NUL, ws=A(10), ws_bytes=BIG, stream=NUL)


@pytest.mark.parametrize("kw,code", ATTN_BAD + [
    (dict(lse=NUL), 1), (dict(do=NUL), 1), (dict(dq=NUL), 1), (dict(dk=NUL), 1), (dict(dv=NUL), 1),
    (dict(dq=A(1)), 1), (dict(dk=A(9)), 1), (dict(dv=A(6, 16)), 1), (dict(do=A(6, 2)), 1), (dict(ws=NUL), 3),
    (dict(ws_bytes=256), 3), (dict(ws=A(10, 16)), 3), (dict(ws=A(7)), 3), (dict(ws=A(2)), 3)])
def test_attn_backward_refusals(lib, kw, code):
    assert _call(lib.pkv_attn_varlen_backward, ATTN_BWD, kw) == code


LIN = dict(q=A(1), k=A(2), v=A(3), g=A(4), cu=P, max_segs=4, N=256, H=4, Dk=64, Dv=64, scale=1.0, dtype=0, s0=A(5),
           o=A(6), fs=A(7), flags=NUL, ws=A(8), ws_bytes=BIG, stream=NUL)
LIN_BAD = [
    (dict(q=NUL), 1), (dict(k=NUL), 1), (dict(v=NUL), 1), (dict(g=NUL), 1), (dict(N=0), 1), (dict(N=1 << 31), 1),
    (dict(H=0), 1), (dict(max_segs=0), 1), (dict(max_segs=1 << 21), 1), (dict(scale=float("nan")), 1),
    (dict(Dk=48), 2), (dict(Dv=256), 2), (dict(dtype=-1), 2), (dict(v=A(3, 8)), 1), (dict(g=A(4, 2)), 1),
    (dict(s0=A(5, 4)), 1),
]


@pytest.mark.parametrize("kw,code", LIN_BAD + [
    (dict(o=NUL), 1), (dict(o=A(1)), 1), (dict(fs=A(5, 4096)), 1), (dict(fs=A(6)), 1), (dict(o=A(6, 2)), 1)])
def test_linear_refusals(lib, kw, code):
    assert _call(lib.pkv_linear_attn_varlen, LIN, kw) == code


LIN_BWD = dict(q=A(1), k=A(2), v=A(3), g=A(4), cu=P, max_segs=4, N=256, H=4, Dk=64, Dv=64, scale=1.0, dtype=0,
               s0=A(5), do=A(6), dF=A(7), dq=A(8), dk=A(9), dv=A(10), di=A(11), flags=NUL, ws=A(12), ws_bytes=BIG,
               stream=NUL)


@pytest.mark.parametrize("kw,code", LIN_BAD + [
    (dict(do=NUL), 1), (dict(dq=NUL), 1), (dict(dk=NUL), 1), (dict(dv=NUL), 1), (dict(dq=A(6)), 1),
    (dict(di=A(7, 1024)), 1), (dict(dv=A(9, 64)), 1), (dict(dF=A(7, 8)), 1)])
def test_linear_backward_refusals(lib, kw, code):
    assert _call(lib.pkv_linear_attn_varlen_backward, LIN_BWD, kw) == code


@pytest.mark.parametrize("bwd", [False, True])
def test_linear_workspace_refusals(lib, bwd):
    size = (lib.pkv_linear_attn_varlen_backward_workspace_size if bwd else lib.pkv_linear_attn_varlen_workspace_size)
    base = dict(LIN_BWD if bwd else LIN, N=65536)
    fn = lib.pkv_linear_attn_varlen_backward if bwd else lib.pkv_linear_attn_varlen
    need = size(65536, 4, 64, 64, 4, 0)
    if need == 0:
        return
    for kw in (dict(ws=NUL), dict(ws_bytes=need - 1), dict(ws=A(12 if bwd else 8, 16))):
        assert _call(fn, base, kw) == 3, kw
    assert _call(fn, base, dict(ws=A(1))) == 1        # overlaps an input


STEP = dict(q=A(1), k=A(2), v=A(3), g=A(4), slots=A(5), R=4, S=8, H=4, Dk=64, Dv=64, scale=1.0, dtype=0, state=A(6),
            o=A(7), flags=NUL, stream=NUL)
STEP_BAD = [
    (dict(q=NUL), 1), (dict(k=NUL), 1), (dict(v=NUL), 1), (dict(g=NUL), 1), (dict(state=NUL), 1), (dict(o=NUL), 1),
    (dict(R=0), 1), (dict(R=(1 << 20) + 1), 1), (dict(S=0), 1), (dict(H=0), 1), (dict(H=65536), 1),
    (dict(slots=NUL, S=3), 1), (dict(scale=float("inf")), 1), (dict(Dk=16), 2), (dict(Dv=96), 2), (dict(dtype=3), 2),
    (dict(o=A(3)), 1), (dict(state=A(6, 4)), 1), (dict(o=A(6, 256)), 1), (dict(slots=A(5, 1)), 1), (dict(q=A(1, 2)), 1),
]


@pytest.mark.parametrize("kw,code", STEP_BAD)
def test_step_refusals(lib, kw, code):
    assert _call(lib.pkv_linear_attn_step, STEP, kw) == code


KDA = dict(q=A(1), k=A(2), v=A(3), g=A(4), beta=A(8), slots=A(5), R=4, S=8, H=4, Dk=64, Dv=64, scale=1.0, dtype=0,
           options=0, state=A(6), o=A(7), flags=NUL, stream=NUL)


@pytest.mark.parametrize("kw,code", STEP_BAD + [(dict(beta=NUL), 1), (dict(options=2), 2), (dict(beta=A(8, 1)), 1)])
def test_kda_step_refusals(lib, kw, code):
    assert _call(lib.pkv_kda_step, KDA, kw) == code


# ------------------------------------------------------------ the binding

B16 = torch.bfloat16


def _z(*shape, dtype=B16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call,err,match", [
    (lambda: pkv.attn_varlen(_z(1, 8, 4, 64), _z(1, 8, 3, 64), _z(1, 8, 3, 64)), ValueError, "multiple"),
    (lambda: pkv.attn_varlen(_z(1, 8, 4, 64), _z(1, 7, 2, 64), _z(1, 7, 2, 64)), ValueError, "k and v"),
    (lambda: pkv.attn_varlen(_z(1, 8, 4, 64), _z(1, 8, 2, 64), _z(1, 8, 4, 64)), ValueError, "k and v"),
    (lambda: pkv.attn_varlen(_z(8, 4, 64), _z(1, 8, 2, 64), _z(1, 8, 2, 64)), ValueError, "4 dims"),
    (lambda: pkv.attn_varlen(_z(1, 8, 4, 64), _z(1, 8, 2, 64, dtype=torch.float32), _z(1, 8, 2, 64)), TypeError, "k"),
    (lambda: pkv.attn_varlen(*[_z(1, 8, 2, 64, dtype=torch.float16)] * 3), TypeError, "unsupported dtype"),
    (lambda: pkv.attn_varlen(_z(1, 8, 4, 128)[..., ::2], _z(1, 8, 2, 64), _z(1, 8, 2, 64)), ValueError, "contiguous"),
    (lambda: pkv.attn_varlen(*[_z(1, 8, 2, 64)] * 3, _z(3, dtype=torch.int64)), TypeError, "cu_seqlens"),
    (lambda: pkv.attn_varlen(*[_z(1, 8, 2, 64)] * 3, _z(1, dtype=torch.int32)), ValueError, "max_segs"),
    (lambda: pkv.attn_varlen(*[_z(1, 8, 2, 64)] * 3, out=_z(1, 8, 2, 32)), ValueError, "out must have shape"),
    (lambda: pkv.attn_varlen(*[_z(1, 8, 2, 64)] * 3), ValueError, "expected a GPU"),
    (lambda: pkv.attn_varlen_backward(*[_z(1, 8, 2, 64)] * 4, _z(8, 2, dtype=torch.float32), _z(1, 8, 2, 64)),
     ValueError, "lse must have shape"),
    (lambda: pkv.attn_varlen_backward(*[_z(1, 8, 2, 64)] * 4, _z(2, 8, dtype=torch.float32), _z(1, 7, 2, 64)),
     ValueError, "do must have shape"),
    (lambda: pkv.chunk_linear_attn_varlen(*[_z(1, 8, 2, 64)] * 3, _z(3, dtype=torch.float32)), ValueError, "g must"),
    (lambda: pkv.chunk_linear_attn_varlen(*[_z(1, 8, 2, 64)] * 3, _z(2)), TypeError, "g has dtype"),
    (lambda: pkv.chunk_linear_attn_varlen(*[_z(1, 8, 2, 64)] * 3, _z(2, dtype=torch.float32),
                                          initial_state=_z(2, 2, 64, 64, dtype=torch.float32)),
     ValueError, "initial_state must have shape"),
    (lambda: pkv.chunk_linear_attn_varlen_backward(*[_z(1, 8, 2, 64)] * 3, _z(2, dtype=torch.float32),
                                                   _z(1, 8, 2, 32)), ValueError, "do must have shape"),
    (lambda: pkv.linear_attn_step(*[_z(3, 2, 64)] * 3, _z(2, dtype=torch.float32),
                                  _z(2, 2, 64, 64, dtype=torch.float32)), ValueError, "3 rows for 2"),
    (lambda: pkv.linear_attn_step(*[_z(3, 2, 64)] * 3, _z(2, dtype=torch.float32),
                                  _z(4, 2, 64, 32, dtype=torch.float32)), ValueError, "state must have shape"),
    (lambda: pkv.linear_attn_step(*[_z(3, 2, 64)] * 3, _z(2, dtype=torch.float32),
                                  _z(4, 2, 64, 64, dtype=torch.float32), _z(2, dtype=torch.int32)),
     ValueError, "slots must have shape"),
    (lambda: pkv.linear_attn_step(*[_z(3, 2, 64)] * 3, _z(2, dtype=torch.float32), _z(4, 2, 64, 64)),
     TypeError, "state has dtype"),
    (lambda: pkv.kda_step(*[_z(3, 2, 64)] * 4, _z(3, 3), _z(4, 2, 64, 64, dtype=torch.float32)),
     ValueError, "beta must have shape"),
])
def test_binding_refusals(call, err, match):
    with pytest.raises(err, match=match):
        call()
