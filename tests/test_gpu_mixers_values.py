"""What single values of a call may and may not reach: rows of the softmax layer go by their own tokens alone, bit
by bit, and hold what the definition gives where values are not finite."""

import numpy as np
import pytest
import torch

import packed_varlen_gated_amd as pkv
from test_gpu_mixers import attn_inputs, cu_gpu

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def forms(N):
    """cu_seqlens of one segment: as the only slot (waves may share queries) and with an empty one behind it."""
    return [None, cu_gpu([0, N, N])]


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("a", [95, 127, 735, 1090])
def test_attn_rows_go_by_their_own_scores(dtype, D, a):
    """A token whose scores leave every range (or are NaN) is the last of a block of queries, past the first tile of
    keys: the rows before it keep their bits, though their own maxima grow in that tile too."""
    N = 1100
    q, k, v, _ = attn_inputs(a, N, 4, 2, D, dtype)
    q[0, a, :, 3] = 1.0
    for cu in forms(N):
        ref, rl = pkv.attn_varlen(q, k, v, cu)
        assert torch.isfinite(ref).all()
        for t, ch, x in (("k", 3, INF), ("k", 3, -INF), ("q", 3, INF), ("q", slice(None), NAN), ("q", 3, 3e4), ("q", 3, -3e4),
                         ("k", slice(None), 3e4)):
            q2, k2 = q.clone(), k.clone()
            (q2 if t == "q" else k2)[0, a, :, ch] = x
            o, lse = pkv.attn_varlen(q2, k2, v, cu)
            assert torch.equal(o[0, :a], ref[0, :a]) and torch.equal(lse[:, :a], rl[:, :a]), (t, x, cu is None)
