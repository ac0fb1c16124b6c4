"""include/pkv_softmax.h without a GPU: what its checks pass and refuse beside the first list (test_softmax_abi.py). No
call here gets past the checks, so nothing is launched."""

import pytest
import torch

import packed_varlen_gated_amd as pkv

from test_mixers_abi import A, BIG, NUL, _call, lib  # noqa: F401
from test_softmax_abi import APPEND, PAGED, ROPE, ROPE_BWD


@pytest.mark.parametrize("sinks", [0, 64, 65, 1000, 2 ** 31 - 1])
def test_sinks_without_a_window_are_ignored(lib, sinks):  # noqa: F811
    """They pass the checks up to the last one, the workspace's; with a window at most 64 do."""
    assert _call(lib.pkv_attn_paged, PAGED, dict(sinks=sinks, ws=NUL)) == 3
    assert _call(lib.pkv_attn_paged, PAGED, dict(sinks=sinks, window=8, ws=NUL)) == (3 if sinks <= 64 else 2)


@pytest.mark.parametrize("stride", [(1 << 40) + 8, 1 << 40, (1 << 40) - 128, 1 << 39, 1 << 38])
def test_strides_whose_bytes_overflow_are_refused(lib, stride):  # noqa: F811
    """Tokens so far apart that N of them pass 64 bits, or any address space; no tensor lies behind another."""
    far = dict(N=1 << 25, q=A(1 << 12), k=A(1 << 13))
    rope = dict(far, qo=A(1 << 8), ko=A(1 << 9))
    back = dict(far, dq=A(1 << 6), dk=A(1 << 7), dqo=A(1 << 8), dko=A(1 << 9))
    append = dict(N=1 << 25, k=A(1 << 12), v=A(1 << 13))
    for name in ("qs", "ks"):
        assert _call(lib.pkv_qk_norm_rope, ROPE, {**rope, name: stride}) == 1
        assert _call(lib.pkv_qk_norm_rope_backward, ROPE_BWD, {**back, name: stride}) == 1
    for name in ("ks", "vs"):
        assert _call(lib.pkv_paged_kv_append, APPEND, {**append, name: stride}) == 1


@pytest.mark.parametrize("D,rows", [(64, 32), (128, 32), (64, 33), (128, 40)])
def test_paged_workspace_goes_by_what_a_request_can_have(lib, D, rows):  # noqa: F811
    """Sums of tiles of 256 rows only where a request can have more than 32: chunks of enough tokens, or many heads."""
    size = lambda N, R, Hq, Hkv: lib.pkv_attn_paged_workspace_size(N, R, Hq, Hkv, D, 0)
    one = size(1, 1, 32, 8)
    assert 0 < one < 18 << 20
    assert all(size(N, R, Hq, Hkv) == one for N, R, Hq, Hkv in ((8, 8, 32, 8), (8, 1, 4, 1), (32, 3, 2, 2), (1, 1, 32, 1)))
    many = size(9, 1, 32, 8)
    assert many > 4 * one
    assert all(size(N, R, Hq, Hkv) == many for N, R, Hq, Hkv in ((64, 64, 32, 8), (33, 1, 5, 5), (1, 1, 33, 1)))
    # the call asks for no more: without cu_seqlens, and with it (a workspace of a byte less is refused before a launch)
    call = dict(PAGED, D=D, Hq=rows, Hkv=1, N=1, R=1, window=8, sinks=64)
    for cu in (NUL, A(5)):
        need = many if rows > 32 else one
        assert _call(lib.pkv_attn_paged, call, dict(cu=cu, ws_bytes=need - 1)) == 3
        assert _call(lib.pkv_attn_paged, call, dict(cu=cu, ws_bytes=need, o=A(9))) == 1  # (the size passes, o overlaps)
    call = dict(PAGED, D=D, Hq=32, Hkv=8, N=64, R=64)
    assert _call(lib.pkv_attn_paged, call, dict(cu=NUL, ws_bytes=one, o=A(9))) == 1
    assert _call(lib.pkv_attn_paged, call, dict(ws_bytes=one, o=A(9))) == 3


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 32), (torch.float32, 128)])
def test_the_binding_s_workspace_size(dtype, D):
    sizes = [pkv.attn_paged_workspace_size(300, 300, 8, 2, D, dtype, chunks=c) for c in (True, False)]
    assert sizes[0] == pkv.attn_paged_workspace_size(300, 300, 8, 2, D, dtype)
    assert (4 * sizes[1] < sizes[0]) if dtype is torch.bfloat16 and D > 32 else sizes[0] == sizes[1]
