"""The bound of mixer_states.py on a CPU form of the kernels' arithmetic: three bf16 parts pass it, two do not."""

import numpy as np
import pytest
import torch

from mixer_states import state_bound


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).float().numpy()


def _state(k, v, g, parts):
    """fp32, in chunks of 32 tokens: carry, then the products of the decayed v's parts token by token."""
    X = np.zeros((k.shape[1], v.shape[1]), dtype=np.float32)
    g2 = np.float32(g * np.log2(np.e))
    for a in range(0, len(k), 32):
        n = min(32, len(k) - a)
        X *= np.exp2(g2 * np.float32(n), dtype=np.float32)
        w = np.exp2(g2 * np.arange(n - 1, -1, -1, dtype=np.float32), dtype=np.float32)
        y = v[a:a + n] * w[:, None]
        for _ in range(parts):
            r = _bf16(y)
            y = y - r
            for s in range(n):
                X += k[a + s][:, None] * r[s][None, :]
    return X


@pytest.mark.parametrize("n,g", [(31, -0.01), (31, -0.3), (300, -0.3), (90, -0.01), (700, -0.05)])
@pytest.mark.parametrize("seed", range(3))
def test_bound_tells_two_parts_from_three(n, g, seed):
    rng = np.random.default_rng(seed)
    k, v = _bf16(rng.standard_normal((n, 64)) / 8), _bf16(rng.standard_normal((n, 64)))
    w = np.exp(g * np.arange(n - 1, -1, -1))
    ref = (k.astype(np.float64) * w[:, None]).T @ v.astype(np.float64)
    rel = [np.linalg.norm(_state(k, v, g, p) - ref) / np.linalg.norm(ref) for p in (3, 2)]
    assert rel[0] <= state_bound(n, g) < rel[1], (rel, state_bound(n, g))
