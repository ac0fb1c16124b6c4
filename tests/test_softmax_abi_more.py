"""include/pkv_softmax.h without a GPU: what its checks pass and refuse beside the first list (test_softmax_abi.py). No
call here gets past the checks, so nothing is launched."""

import pytest

from test_mixers_abi import A, BIG, NUL, _call, lib  # noqa: F401
from test_softmax_abi import PAGED


@pytest.mark.parametrize("sinks", [0, 64, 65, 1000, 2 ** 31 - 1])
def test_sinks_without_a_window_are_ignored(lib, sinks):  # noqa: F811
    """They pass the checks up to the last one, the workspace's; with a window at most 64 do."""
    assert _call(lib.pkv_attn_paged, PAGED, dict(sinks=sinks, ws=NUL)) == 3
    assert _call(lib.pkv_attn_paged, PAGED, dict(sinks=sinks, window=8, ws=NUL)) == (3 if sinks <= 64 else 2)
