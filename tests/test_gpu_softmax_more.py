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


@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
def test_paged_an_infinity_stays_one_under_larger_scores(dtype, D):
    """A weight of e^-300 is none in fp32, but more than 0: an infinite value that it stands at is the sum, whether its
    key is walked before or after the larger scores."""
    rng = np.random.default_rng(D)
    n = 1000
    for news, at in ((1, 5), (1, 990), (40, 5)):
        table, kp, vp = cache_of(rng, [n], 16, 1, D, dtype)
        q = on_gpu(rng.standard_normal((1, 1, D)), dtype)
        for p in [*range(39, 960, 32)] + [at]:       # in every tile of keys
            x = q[0, 0].float()
            kp[int(table[0, p // 16]), p % 16, 0] = (x * ((0.0 if p == at else 300.0) / float(x @ x))).to(kp.dtype)
        args = (i32(table), i32([n]), i32([0, news]))
        q = q.expand(news, 2, D).contiguous()
        want, wl = pkv.attn_paged(q, kp, vp, *args, scale=1.0, output_lse=True)
        assert float(wl.min()) > 290
        bad = torch.tensor([float("inf"), -float("inf"), float("nan")])
        v2 = vp.clone()
        v2[int(table[0, at // 16]), at % 16, 0, 3:6] = bad.to(v2)
        o, lse = pkv.attn_paged(q, kp, v2, *args, scale=1.0, output_lse=True)
        assert torch.equal(lse, wl)
        hit = torch.zeros(D, dtype=torch.bool, device=dev())
        hit[3:6] = True
        assert torch.equal(o[..., ~hit], want[..., ~hit])
        got = torch.nan_to_num(o[..., hit].float().cpu(), 7.0, 8.0, 9.0)
        assert torch.equal(got, torch.nan_to_num(bad, 7.0, 8.0, 9.0).expand_as(got)), (news, at, o[..., hit])


@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
@pytest.mark.parametrize("Hq,Hkv,news", [(8, 2, None), (40, 1, None), (8, 2, [1, 0, 4, 3]), (8, 2, [1, 0, 40, 3])])
def test_paged_takes_no_more_than_its_workspace(dtype, D, Hq, Hkv, news):
    """A workspace of just the size that the call asks for: the same bits as with its own, and nothing behind it changes."""
    rng = np.random.default_rng(D)
    lens = [3000, 17, 900, 2100]
    cu = None if news is None else i32(np.concatenate([[0], np.cumsum(news)]))
    N = sum(news or [1] * 4)
    table, kp, vp = cache_of(rng, lens, 16, Hkv, D, dtype)
    q = on_gpu(rng.standard_normal((N, Hq, D)), dtype)
    need = pkv.attn_paged_workspace_size(N, 4, Hq, Hkv, D, q.dtype, chunks=news is not None)
    args = (q, kp, vp, i32(table), i32(lens), cu)
    want, wl = pkv.attn_paged(*args, output_lse=True)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=dev())
    for _ in range(2):
        o, lse = pkv.attn_paged(*args, output_lse=True, workspace=ws[:need]) if need else (want, wl)
        assert torch.equal(o, want) and torch.equal(lse, wl) and bool((ws[need:] == 255).all())
    if need:
        with pytest.raises(ValueError, match="workspace holds"):
            pkv.attn_paged(*args, workspace=ws[:need - 1])
