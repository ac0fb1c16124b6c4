"""The softmax layer's kernels on the GPU: calls that the documentation allows and that are easily answered wrongly."""

import numpy as np
import pytest
import torch

import packed_varlen_gated_amd as pkv
from oracle import softmax
from test_gpu_mixers import dev, on_gpu
from test_gpu_softmax import PAGED_TYPES, cache_of, i32

pytestmark = pytest.mark.gpu


def pages_in_use(lens, news, size, window, sinks, width):
    """[R, width]: whether a new token of the request sees a place of the page."""
    use = np.zeros((len(lens), width), dtype=bool)
    for r, (n, new) in enumerate(zip(lens, news)):
        at = np.arange(n)
        use[r, at[softmax.visible(np.arange(n - new, n), at, window, sinks).any(0)] // size] = True
    return use


@pytest.mark.parametrize("size", [16, 48])
@pytest.mark.parametrize("window,sinks", [(20, 0), (20, 4), (33, 17), (16, 64), (1, 0), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
def test_paged_entries_that_no_token_needs_may_hold_anything(dtype, D, window, sinks, size):
    """Pages behind the window and past the sinks are gone from the table: no flag, and the same bits."""
    rng = np.random.default_rng(window % 97)
    for lens, news in (([101, 700, 33, 16, 65, 0], [1] * 6), ([101, 700, 333, 40, 0], [7, 130, 33, 1, 0])):
        cu = None if news == [1] * len(lens) else i32(np.concatenate([[0], np.cumsum(news)]))
        table, kp, vp = cache_of(rng, lens, size, 2, D, dtype)
        q = on_gpu(rng.standard_normal((sum(news), 4, D)), dtype)
        use = pages_in_use(lens, news, size, window, sinks, table.shape[1])
        flags = torch.zeros(1, dtype=torch.int32, device=dev())
        call = lambda t: pkv.attn_paged(q, kp, vp, i32(t), i32(lens), cu, window, sinks, output_lse=True, flags=flags)
        want, wl = call(table)
        for gone in (-1, 1 << 30, -(1 << 31)):
            o, lse = call(np.where(use, table, gone))
            assert int(flags) == 0
            assert torch.equal(o, want) and torch.equal(lse, wl)
        # one that is needed still sets the flag
        r = int(np.flatnonzero(use.any(1))[0])
        for at in {int(np.flatnonzero(use[r])[0]), int(np.flatnonzero(use[r])[-1])}:
            t = table.copy()
            t[r, at] = -1
            call(t)
            assert int(flags) == pkv.FLAG_BAD_PAGE
            flags.zero_()
