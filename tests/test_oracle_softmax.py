"""Pins of the softmax layer's oracle (oracle/softmax.py): brute force, complex
numbers, the unwindowed oracle, and central finite differences of every gradient."""

import cmath
import math

import numpy as np
import pytest

from oracle import mixers, softmax
from test_oracle_mixers import CU, _differences, _rng


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 1), (2, 4), (50, 0)])
def test_window_brute_force(window, sinks):
    q, k, v = _rng(0, (13, 4, 3), (13, 2, 3), (13, 2, 3))
    o, lse = softmax.attn_window_varlen(q, k, v, window, sinks, CU, 0.7)
    for t in range(13):
        seg = [i for i in range(4) if CU[i] <= t < CU[i + 1]]
        for h in range(4):
            if not seg:
                assert not o[t, h].any() and lse[h, t] == -np.inf
                continue
            a = int(CU[seg[0]])
            keys = [s for s in range(a, t + 1) if t - s < window or s - a < sinks]
            w = [math.exp(0.7 * sum(q[t, h, d] * k[s, h // 2, d] for d in range(3))) for s in keys]
            z = math.fsum(w)
            for d in range(3):
                assert abs(o[t, h, d] - math.fsum(x / z * v[s, h // 2, d] for x, s in zip(w, keys))) < 1e-13
            assert abs(lse[h, t] - math.log(z)) < 1e-13


def test_a_wide_window_is_none():
    q, k, v, do = _rng(1, (11, 4, 3), (11, 2, 3), (11, 2, 3), (11, 4, 3))
    for got, want in zip(softmax.attn_window_varlen(q, k, v, 11, 0, CU), mixers.attn_varlen(q, k, v, CU)):
        np.testing.assert_allclose(got, want, rtol=1e-13)
    for got, want in zip(softmax.attn_window_varlen_backward(q, k, v, do, 1, 11, CU),
                         mixers.attn_varlen_backward(q, k, v, do, CU)):
        np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("window,sinks", [(2, 0), (2, 1), (4, 2)])
def test_window_gradients_by_differences(name, window, sinks):
    q, k, v, do = _rng(7, (11, 4, 3), (11, 2, 3), (11, 2, 3), (11, 4, 3))
    grads = dict(zip("qkv", softmax.attn_window_varlen_backward(q, k, v, do, window, sinks, CU, 0.7)))
    _differences(dict(q=q, k=k, v=v), name, grads[name], lambda x: float(
        (softmax.attn_window_varlen(x["q"], x["k"], x["v"], window, sinks, CU, 0.7)[0] * do).sum()))


def _cache(rng, lens, size, Hkv, D, spare=2):
    need = [-(-n // size) for n in lens]
    pages = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), -1)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = pages[at:at + n]
        at += n
    return table, np.full((len(pages), size, Hkv, D), np.nan), np.full((len(pages), size, Hkv, D), np.nan)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2)])
def test_a_cache_filled_in_chunks_is_the_packed_attention(window, sinks):
    rng = np.random.default_rng(3)
    lens = [7, 1, 0, 12]
    q, k, v = (rng.standard_normal((20, h, 3)) for h in (4, 2, 2))
    cu = np.concatenate([[0], np.cumsum(lens)])
    if window:
        want = softmax.attn_window_varlen(q, k, v, window, sinks, cu)
    else:
        want = mixers.attn_varlen(q, k, v, cu)
    table, kp, vp = _cache(rng, lens, 4, 2, 3)
    done = np.zeros(4, dtype=int)
    for step in ([3, 1, 0, 5], [1, 0, 0, 1], [3, 0, 0, 6]):
        c = np.concatenate([[0], np.cumsum(step)])
        idx = np.concatenate([cu[r] + done[r] + np.arange(n) for r, n in enumerate(step)])
        done += step
        kp, vp = softmax.paged_kv_append(k[idx], v[idx], kp, vp, table, done, c)
        o, lse = softmax.attn_paged(q[idx], kp, vp, table, done, c, window, sinks)
        np.testing.assert_allclose(o, want[0][idx], rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(lse, want[1][:, idx], rtol=1e-12, atol=1e-14)
    idle, _ = softmax.attn_paged(q[:4], kp, vp, table, [7, 0, 0, 12])   # one token each, two of them idle
    assert not idle[1:3].any() and idle[0].any() and np.isfinite(idle).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_as_complex_numbers(interleaved):
    x, w = _rng(4, (5, 2, 8), (8,))
    pos, freq = np.array([0, 3, -1, 70, 100000]), np.array([1.0, 0.01])
    y = softmax.norm_rope(x, w, pos, freq, 1e-3, interleaved)
    for n in range(5):
        for h in range(2):
            if pos[n] < 0:
                assert not y[n, h].any()
                continue
            u = w * x[n, h] / math.sqrt((x[n, h] ** 2).mean() + 1e-3)
            np.testing.assert_allclose(y[n, h, 4:], u[4:], rtol=1e-14)
            for i in range(2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 2)
                z = complex(u[a], u[b]) * cmath.exp(1j * pos[n] * freq[i])
                # 1e-10: the plain fp64 angle is off by 2^-53 of itself, up to 1e5 of them
                assert abs(y[n, h, a] - z.real) < 1e-10 and abs(y[n, h, b] - z.imag) < 1e-10


def test_angles_of_the_farthest_positions():
    pos, f = 2 ** 31 - 1, np.float32(0.7).astype(np.float64)
    from fractions import Fraction
    turn = Fraction(2) * Fraction("3.14159265358979323846264338327950288419716939937510")
    exact = Fraction(pos) * Fraction(float(f))
    rest = float(exact - round(exact / turn) * turn)
    # the product is exact in 64 bits; a turn's rounding counts 2.4e8 times: 2.4e8 * 2^-64 * 8 < 2e-10
    assert abs(softmax.angles([pos], [f])[0, 0] - rest) < 2e-10


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ["x", "w"])
def test_norm_rope_gradients_by_differences(name, interleaved):
    x, w, dy = _rng(5, (5, 2, 8), (8,), (5, 2, 8))
    pos, freq = np.array([0, 3, -1, 70, 1000]), np.array([1.0, 0.1])
    dx, dw = softmax.norm_rope_backward(x, dy, w, pos, freq, 1e-3, interleaved)
    _differences(dict(x=x, w=w), name, dict(x=dx, w=dw)[name], lambda z: float(
        (softmax.norm_rope(z["x"], z["w"], pos, freq, 1e-3, interleaved) * dy).sum()))
