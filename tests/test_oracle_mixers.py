"""Pins of the mixers' oracle (oracle/mixers.py): brute force, closed forms, KDA
with a broadcast gate, and central finite differences of every gradient."""

import math

import numpy as np
import pytest

import oracle
from oracle import mixers

CU = np.array([0, 1, 4, 4, 11])


def _rng(seed, *shapes):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in shapes]


def test_attn_brute_force():
    q, k, v = _rng(0, (13, 4, 3), (13, 2, 3), (13, 2, 3))
    o, lse = mixers.attn_varlen(q, k, v, CU, 0.7)
    for t in range(13):
        seg = [i for i in range(4) if CU[i] <= t < CU[i + 1]]
        for h in range(4):
            if not seg:
                assert not o[t, h].any() and lse[h, t] == -np.inf
                continue
            keys = range(int(CU[seg[0]]), t + 1)
            w = [math.exp(0.7 * sum(q[t, h, d] * k[s, h // 2, d] for d in range(3))) for s in keys]
            z = math.fsum(w)
            for d in range(3):
                want = math.fsum(x / z * v[s, h // 2, d] for x, s in zip(w, keys))
                assert abs(o[t, h, d] - want) < 1e-13
            assert abs(lse[h, t] - math.log(z)) < 1e-13


def test_attn_closed_forms():
    q, k, v = _rng(1, (9, 2, 4), (9, 2, 4), (9, 2, 4))
    o, _ = mixers.attn_varlen(q, k, v, np.arange(10))          # one key each
    assert np.array_equal(o, v)
    o, lse = mixers.attn_varlen(q * 0, k, v)                   # equal scores: running means
    # atol: two sums of at most 9 terms below 4 in another order, 2 * 9 * 4 * 2^-53 < 1e-14
    np.testing.assert_allclose(o, np.cumsum(v, 0) / np.arange(1, 10)[:, None, None], rtol=1e-13, atol=1e-14)
    np.testing.assert_allclose(lse[0], np.log(np.arange(1, 10)), rtol=1e-13, atol=1e-15)


def test_linear_closed_forms():
    q, k, v = _rng(2, (11, 2, 3), (11, 2, 3), (11, 2, 5))
    g = np.array([-0.3, 0.0])
    o, fs = mixers.linear_attn_varlen(q, k, v, g, CU, 0.5)
    for i in range(4):
        for t in range(CU[i], CU[i + 1]):
            for h in range(2):
                want = sum(math.exp(g[h] * (t - s)) * (q[t, h] @ k[s, h]) * v[s, h] for s in range(CU[i], t + 1))
                np.testing.assert_allclose(o[t, h], 0.5 * want, rtol=1e-12, atol=1e-13)
    ones = np.ones((6, 1, 1))
    o, fs = mixers.linear_attn_varlen(ones, ones, ones, np.array([math.log(0.5)]))
    np.testing.assert_allclose(o[:, 0, 0], 2 - 0.5 ** np.arange(6), rtol=1e-14)    # geometric series
    assert fs[0, 0, 0, 0] == o[-1, 0, 0]


def test_linear_is_kda_with_one_gate():
    q, k, v, S0 = _rng(3, (11, 2, 3), (11, 2, 3), (11, 2, 5), (4, 2, 3, 5))
    g = np.array([-0.3, -0.01])
    gates = np.broadcast_to(g[None, :, None], (11, 2, 3))
    o, fs = mixers.linear_attn_varlen(q, k, v, g, CU, 0.5, S0)
    ro, rfs = oracle.chunk_kda_varlen(q, k, v, gates, np.ones((11, 2)), CU, 0.5, initial_state=S0)
    np.testing.assert_allclose(o, ro, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(fs, rfs, rtol=1e-13, atol=1e-13)


def test_step_is_the_recurrence():
    q, k, v, S0 = _rng(4, (3, 2, 3), (3, 2, 3), (3, 2, 5), (6, 2, 3, 5))
    gates = -np.abs(_rng(5, (3, 2, 3))[0])
    beta = np.abs(_rng(6, (3, 2))[0])
    o, S = mixers.step(q, k, v, np.exp(gates), beta, S0, [4, -1, 4], 0.5)
    ro, rfs = oracle.chunk_kda_varlen(q[:1], k[:1], v[:1], gates[:1], beta[:1], None, 0.5, initial_state=S0[4:5])
    np.testing.assert_allclose(o[0], ro[0], rtol=1e-13)
    np.testing.assert_allclose(S[4], rfs[0], rtol=1e-13)
    assert not o[1].any() and not o[2].any() and np.array_equal(S[:4], S0[:4]) and np.array_equal(S[5], S0[5])


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_attn_gradients_by_differences(name):
    q, k, v, do = _rng(7, (11, 4, 3), (11, 2, 3), (11, 2, 3), (11, 4, 3))
    grads = dict(zip("qkv", mixers.attn_varlen_backward(q, k, v, do, CU, 0.7)))
    _differences(dict(q=q, k=k, v=v), name, grads[name],
                 lambda x: float((mixers.attn_varlen(x["q"], x["k"], x["v"], CU, 0.7)[0] * do).sum()))


@pytest.mark.parametrize("name", ["q", "k", "v", "S0"])
def test_linear_gradients_by_differences(name):
    q, k, v, do, S0, dF = _rng(8, (11, 2, 3), (11, 2, 3), (11, 2, 5), (11, 2, 5), (4, 2, 3, 5), (4, 2, 3, 5))
    g = np.array([-0.3, -0.01])
    grads = dict(zip(("q", "k", "v", "S0"), mixers.linear_attn_varlen_backward(q, k, v, g, do, CU, 0.7, S0, dF)))

    def loss(x):
        o, fs = mixers.linear_attn_varlen(x["q"], x["k"], x["v"], g, CU, 0.7, x["S0"])
        return float((o * do).sum() + (fs * dF).sum())
    _differences(dict(q=q, k=k, v=v, S0=S0), name, grads[name], loss)


def _differences(ins, name, grad, loss, h=1e-5):
    rng = np.random.default_rng(9)
    for _ in range(12):
        d = rng.standard_normal(ins[name].shape)
        up, dn = dict(ins), dict(ins)
        up[name], dn[name] = ins[name] + h * d, ins[name] - h * d
        want = (loss(up) - loss(dn)) / (2 * h)
        got = float((grad * d).sum())
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want)), (got, want)
