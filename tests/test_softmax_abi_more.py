"""include/pkv_softmax.h without a GPU: what its checks pass and refuse beside the first list (test_softmax_abi.py). No
call here gets past the checks, so nothing is launched."""

import pytest

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
