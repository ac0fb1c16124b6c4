"""include/pkv_softmax.h without a GPU: every declared function is exported, and bad
arguments are refused, by the library and by the binding, before anything is launched."""

import os
import re

import pytest
import torch

import packed_varlen_gated_amd as pkv
from conftest import ROOT
from test_mixers_abi import A, ATTN, ATTN_BAD, ATTN_BWD, B16, BIG, NUL, P, _call, _z, lib  # noqa: F401


def test_exports_every_declared_function(lib):  # noqa: F811
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pkv_softmax.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pkv_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 9, names
    for n in names:
        assert hasattr(lib, n), n


def test_flags_are_distinct():
    assert pkv.FLAG_BAD_PAGE == 32 and pkv.FLAG_BAD_LENGTH == 64 and pkv.FLAG_BAD_SLOT == 16


ROPE = dict(q=A(1), k=A(2), qs=256, ks=128, wq=A(3), wk=A(4), pos=A(5), freq=A(6), N=64, Hq=4, Hkv=2, D=64, rot=64,
            eps=1e-6, dtype=0, options=0, qo=A(7), ko=A(8), stream=NUL)
ROPE_BAD = [
    (dict(q=NUL), 1), (dict(k=NUL), 1), (dict(N=0), 1), (dict(N=(1 << 25) + 1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1),
    (dict(Hq=65537), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(D=96), 2), (dict(rot=8), 2), (dict(rot=80), 2), (dict(rot=-16), 2), (dict(dtype=2), 2), (dict(options=1), 2),
    (dict(qs=255), 1), (dict(ks=120), 1), (dict(qs=260), 1), (dict(ks=-128), 1), (dict(freq=NUL), 1),
    (dict(q=A(1, 8)), 1), (dict(k=A(2, 2)), 1), (dict(wq=A(3, 2)), 1), (dict(pos=A(5, 1)), 1), (dict(freq=A(6, 3)), 1),
]


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(qo=NUL), 1), (dict(ko=NUL), 1), (dict(qo=A(1)), 1), (dict(qo=A(7, 8)), 1), (dict(ko=A(7, 64)), 1),
    (dict(qo=A(1, 64 * 512 - 16)), 1), (dict(qs=2048, qo=A(1, 63 * 4096)), 1), (dict(ko=A(3)), 1)])
def test_norm_rope_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_qk_norm_rope, ROPE, kw) == code


ROPE_BWD = dict(q=A(1), k=A(2), qs=256, ks=128, dqo=A(9), dko=A(10), wq=A(3), wk=A(4), pos=A(5), freq=A(6), N=64, Hq=4,
                Hkv=2, D=64, rot=64, eps=1e-6, dtype=0, options=0, dq=A(7), dk=A(8), dwq=A(11), dwk=A(12), ws=A(13),
                ws_bytes=BIG, stream=NUL)


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(dq=NUL), 1), (dict(dk=NUL), 1), (dict(dqo=NUL), 1), (dict(dko=NUL), 1), (dict(dq=A(9)), 1),
    (dict(dk=A(10, 32)), 1), (dict(dwq=A(11, 1)), 1), (dict(dwk=A(11, 128)), 1), (dict(dqo=A(9, 4)), 1),
    (dict(ws=NUL), 3), (dict(ws_bytes=64), 3), (dict(ws=A(13, 16)), 3), (dict(ws=A(2)), 1)])
def test_norm_rope_backward_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_qk_norm_rope_backward, ROPE_BWD, kw) == code


def _window(base, window=16, sinks=2):
    d = {}
    for n, x in base.items():
        d[n] = x
        if n == "dtype":
            d.update(window=window, sinks=sinks)
    return d


WIN_BAD = ATTN_BAD + [(dict(window=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(sinks=65), 2)]


@pytest.mark.parametrize("kw,code", WIN_BAD + [
    (dict(o=NUL), 1), (dict(o=A(1, 64)), 1), (dict(o=A(3)), 1), (dict(o=A(4, 4)), 1), (dict(lse=A(5, 2)), 1),
    (dict(lse=A(4, 64)), 1), (dict(flags=A(4)), 1)])
def test_window_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_attn_window_varlen, _window(ATTN), kw) == code


@pytest.mark.parametrize("kw,code", WIN_BAD + [
    (dict(lse=NUL), 1), (dict(do=NUL), 1), (dict(dq=NUL), 1), (dict(dk=NUL), 1), (dict(dv=NUL), 1),
    (dict(dq=A(1)), 1), (dict(dk=A(9)), 1), (dict(dv=A(6, 16)), 1), (dict(do=A(6, 2)), 1), (dict(ws=NUL), 3),
    (dict(ws_bytes=256), 3), (dict(ws=A(10, 16)), 3), (dict(ws=A(7)), 3), (dict(ws=A(2)), 3)])
def test_window_backward_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_attn_window_varlen_backward, _window(ATTN_BWD), kw) == code


@pytest.mark.parametrize("window,sinks", [(1, 1), (63, 4), (64, 4), (127, 2), (300, 64), (5000, 1)])
def test_window_workspace_holds_every_far_chunk(lib, window, sinks):  # noqa: F811
    """8 sinks D Hkv bytes for every chunk of queries behind a segment's window, wherever the segments lie."""
    base = dict(N=20000, Hq=4, Hkv=2, D=64, max_segs=30, dtype=0)
    size = lambda s: lib.pkv_attn_window_varlen_backward_workspace_size(*base.values(), window, s)
    per = 8 * sinks * 64 * 2
    chunk = min(512, base["N"] * 2 // 512 // 128 * 128 + 128)
    chunk = chunk if window < 64 else min(chunk, window)
    most = base["N"] // chunk + (base["max_segs"] if window < 64 else 0)
    assert size(sinks) - size(0) == most * per


APPEND = dict(k=A(1), v=A(2), ks=128, vs=128, table=A(3), lens=A(4), cu=A(5), N=8, R=8, Hkv=2, D=64, size=16, pages=64,
              width=8, dtype=0, kp=A(6), vp=A(7), flags=NUL, stream=NUL)
CACHE_BAD = [
    (dict(table=NUL), 1), (dict(lens=NUL), 1), (dict(N=0), 1), (dict(N=1 << 31), 1), (dict(R=0), 1),
    (dict(cu=NUL, N=7), 1), (dict(Hkv=0), 1), (dict(Hkv=65537), 1), (dict(D=80), 2), (dict(size=8), 2),
    (dict(size=24), 2), (dict(size=0), 2), (dict(size=-16), 2), (dict(size=1 << 17), 2), (dict(pages=0), 1),
    (dict(width=0), 1), (dict(pages=1 << 27), 1), (dict(width=1 << 27), 1), (dict(dtype=7), 2),
    (dict(kp=NUL), 1), (dict(vp=NUL), 1), (dict(kp=A(6, 8)), 1), (dict(table=A(3, 2)), 1), (dict(lens=A(4, 1)), 1),
]


@pytest.mark.parametrize("kw,code", CACHE_BAD + [
    (dict(k=NUL), 1), (dict(v=NUL), 1), (dict(kp=A(7)), 1), (dict(kp=A(1)), 1), (dict(ks=64), 1), (dict(vs=132), 1),
    (dict(v=A(2, 2)), 1), (dict(vp=A(3)), 1), (dict(flags=A(6)), 1)])
def test_append_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_paged_kv_append, APPEND, kw) == code


PAGED = dict(q=A(1), kp=A(6), vp=A(7), table=A(3), lens=A(4), cu=A(5), N=8, R=8, Hq=4, Hkv=2, D=64, size=16, pages=64,
             width=8, scale=1.0, dtype=0, window=0, sinks=0, o=A(2), lse=A(8), flags=NUL, ws=A(9), ws_bytes=BIG,
             stream=NUL)


@pytest.mark.parametrize("kw,code", CACHE_BAD + [
    (dict(q=NUL), 1), (dict(o=NUL), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(scale=float("nan")), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(sinks=65, window=8), 2), (dict(o=A(1)), 1), (dict(o=A(6, 64)), 1),
    (dict(lse=A(2, 16)), 1), (dict(lse=A(8, 2)), 1), (dict(flags=A(2)), 1), (dict(N=1 << 24, Hq=64), 1)])
def test_paged_refusals(lib, kw, code):  # noqa: F811
    assert _call(lib.pkv_attn_paged, PAGED, kw) == code


# ------------------------------------------------------------ the binding

F32, I32 = torch.float32, torch.int32
Q4, K4 = (lambda: _z(1, 8, 4, 64)), (lambda: _z(1, 8, 2, 64))
CACHE = (lambda: (_z(6, 16, 2, 64), _z(6, 16, 2, 64)))


@pytest.mark.parametrize("call,err,match", [
    (lambda: pkv.qk_norm_rope(_z(8, 4, 64), K4()), ValueError, "4 dims"),
    (lambda: pkv.qk_norm_rope(Q4(), _z(1, 7, 2, 64)), ValueError, "k must have shape"),
    (lambda: pkv.qk_norm_rope(Q4(), _z(1, 8, 2, 64, dtype=F32)), TypeError, "k has dtype"),
    (lambda: pkv.qk_norm_rope(_z(1, 8, 4, 128)[..., ::2], K4()), ValueError, "heads of a token"),
    (lambda: pkv.qk_norm_rope(_z(1, 8, 64, 4).transpose(2, 3), K4()), ValueError, "heads of a token"),
    (lambda: pkv.qk_norm_rope(_z(2, 8, 4, 64)[:, :4], _z(2, 4, 2, 64)), ValueError, "equally far"),
    (lambda: pkv.qk_norm_rope(_z(1, 8, 4, 64, dtype=torch.float16), K4()), TypeError, "unsupported dtype"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), _z(32, dtype=F32)), ValueError, "q_weight must have shape"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), None, _z(64)), TypeError, "k_weight has dtype"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), positions=_z(7, dtype=I32)), ValueError, "positions must hold 8"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), positions=_z(8, dtype=torch.int64)), TypeError, "positions has dtype"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), inv_freq=_z(40, dtype=F32)), ValueError, "rot_dim"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), inv_freq=_z(4, dtype=F32)), ValueError, "rot_dim"),
    (lambda: pkv.qk_norm_rope(Q4(), K4(), out=(Q4(), Q4())), ValueError, "k_out must have shape"),
    (lambda: pkv.qk_norm_rope(Q4(), K4()), ValueError, "expected a GPU"),
    (lambda: pkv.qk_norm_rope_backward(Q4(), K4(), K4(), K4()), ValueError, "dq_out must have shape"),
    (lambda: pkv.qk_norm_rope_backward(Q4(), K4(), Q4(), _z(1, 8, 2, 128)[..., :64]), ValueError, "contiguous"),
    (lambda: pkv.attn_window_varlen(Q4(), _z(1, 8, 3, 64), _z(1, 8, 3, 64), 4), ValueError, "multiple"),
    (lambda: pkv.attn_window_varlen(Q4(), K4(), K4(), 1 << 31), ValueError, "window is out of range"),
    (lambda: pkv.attn_window_varlen(Q4(), K4(), K4(), 4, out=K4()), ValueError, "out must have shape"),
    (lambda: pkv.attn_window_varlen(Q4(), K4(), K4(), 4), ValueError, "expected a GPU"),
    (lambda: pkv.attn_window_varlen_backward(Q4(), K4(), K4(), Q4(), _z(8, 4, dtype=F32), Q4(), 4), ValueError,
     "lse must have shape"),
    (lambda: pkv.paged_kv_append(_z(3, 2, 64), _z(3, 2, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)),
     ValueError, "need cu_seqlens"),
    (lambda: pkv.paged_kv_append(_z(2, 2, 64), _z(2, 2, 32), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)),
     ValueError, "v must have shape"),
    (lambda: pkv.paged_kv_append(_z(2, 3, 64), _z(2, 3, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)),
     ValueError, "k_pages and v_pages"),
    (lambda: pkv.paged_kv_append(_z(2, 2, 64), _z(2, 2, 64), *CACHE(), _z(2, 4, dtype=I32), _z(3, dtype=I32)),
     ValueError, "kv_lens must have shape"),
    (lambda: pkv.paged_kv_append(_z(2, 2, 64), _z(2, 2, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32),
                                 _z(4, dtype=I32)), ValueError, "cu_seqlens must have shape"),
    (lambda: pkv.paged_kv_append(_z(2, 2, 64), _z(2, 2, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)),
     ValueError, "expected a GPU"),
    (lambda: pkv.attn_paged(_z(2, 3, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)), ValueError, "divisor"),
    (lambda: pkv.attn_paged(_z(2, 4, 64), *CACHE(), _z(2, 4), _z(2, dtype=I32)), TypeError, "page_table has dtype"),
    (lambda: pkv.attn_paged(_z(2, 4, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32), window=0), ValueError,
     "window must be"),
    (lambda: pkv.attn_paged(_z(2, 4, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32), out=_z(2, 2, 64)),
     ValueError, "out must have shape"),
    (lambda: pkv.attn_paged(_z(2, 4, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32), flags=_z(2, dtype=I32)),
     ValueError, "flags must have shape"),
    (lambda: pkv.attn_paged(_z(2, 4, 64), *CACHE(), _z(2, 4, dtype=I32), _z(2, dtype=I32)), ValueError,
     "expected a GPU"),
])
def test_binding_refusals(call, err, match):
    with pytest.raises(err, match=match):
        call()
