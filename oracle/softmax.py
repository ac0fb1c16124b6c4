"""fp64 oracle of what stands around the packed causal attention: norms of queries
and keys with the rotation by position, attention through a sliding window with
visible first tokens, the paged cache and attention of new tokens over it.

Written from the definitions: ``visible`` says which places a query sees, and every
attention here is one softmax over it. The reverse passes walk the chain rule.

Pinned (tests/test_oracle_softmax.py): brute force over pairs in plain Python,
rotations as complex numbers, the unwindowed oracle, central finite differences of
every gradient.
"""

import numpy as np


def visible(tq, tk, window=0, sinks=0):
    """[len(tq), len(tk)]: whether the query at place tq sees the key at place tk."""
    gap = np.asarray(tq)[:, None] - np.asarray(tk)[None, :]
    see = gap >= 0
    if window > 0:
        see &= (gap < window) | (np.asarray(tk)[None, :] < sinks)
    return see


def weights(q, k, see, scale):
    """Softmax weights [n, m] and ln of their sum [n]; a row that sees nothing has weights of 0 and -inf."""
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = np.where(see.any(1), s.max(1, initial=-np.inf), 0.0)[:, None]
    p = np.where(see, np.exp(s - m), 0.0)
    z = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(z))[:, 0]
    return p / np.where(z > 0, z, 1.0), lse


def _segments(cu, N):
    return [(0, N)] if cu is None else list(zip(cu[:-1].tolist(), cu[1:].tolist()))


def attn_window_varlen(q, k, v, window, sinks=0, cu=None, scale=None):
    """q [N, Hq, D], k and v [N, Hkv, D] -> (o [N, Hq, D], lse [Hq, N])."""
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    o, lse = np.zeros((N, Hq, D)), np.full((Hq, N), -np.inf)
    for a, e in _segments(cu, N):
        see = visible(np.arange(e - a), np.arange(e - a), window, sinks)
        for h in range(Hq if e > a else 0):
            p, lse[h, a:e] = weights(q[a:e, h], k[a:e, h // rep], see, scale)
            o[a:e, h] = p @ v[a:e, h // rep]
    return o, lse


def attn_window_varlen_backward(q, k, v, do, window, sinks=0, cu=None, scale=None):
    """(dq, dk, dv) of sum(o * do)."""
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, e in _segments(cu, N):
        see = visible(np.arange(e - a), np.arange(e - a), window, sinks)
        for h in range(Hq if e > a else 0):
            g = h // rep
            p, _ = weights(q[a:e, h], k[a:e, g], see, scale)
            dp = do[a:e, h] @ v[a:e, g].T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            dq[a:e, h] = scale * ds @ k[a:e, g]
            dk[a:e, g] += scale * ds.T @ q[a:e, h]
            dv[a:e, g] += p.T @ do[a:e, h]
    return dq, dk, dv


def places(table, length, page_size):
    """Where a request's tokens lie: rows of the flattened cache."""
    i = np.arange(length)
    return table[i // page_size].astype(np.int64) * page_size + i % page_size


def paged_kv_append(k, v, k_pages, v_pages, table, lens, cu=None):
    """Copies of the caches with the new tokens in their places."""
    kp, vp = k_pages.copy(), v_pages.copy()
    size = kp.shape[1]
    for r, (a, e) in enumerate(_segments(np.arange(len(lens) + 1) if cu is None else cu, len(k))):
        for t in range(a, e):
            p = int(lens[r]) - (e - t)
            if p >= 0:
                kp[table[r, p // size], p % size] = k[t]
                vp[table[r, p // size], p % size] = v[t]
    return kp, vp


def attn_paged(q, k_pages, v_pages, table, lens, cu=None, window=0, sinks=0, scale=None):
    """q [N, Hq, D] -> (o, lse [Hq, N])."""
    N, Hq, D = q.shape
    size, Hkv = k_pages.shape[1:3]
    rep = Hq // Hkv
    scale = 1 / np.sqrt(D) if scale is None else scale
    o, lse = np.zeros((N, Hq, D)), np.full((Hq, N), -np.inf)
    for r, (a, e) in enumerate(_segments(np.arange(len(lens) + 1) if cu is None else cu, N)):
        n = int(lens[r])
        at = places(table[r], n, size)
        see = visible(np.arange(n - (e - a), n), np.arange(n), window, sinks)
        for h in range(Hq if e > a else 0):
            k, v = (x.reshape(-1, Hkv, D)[at, h // rep] for x in (k_pages, v_pages))
            p, lse[h, a:e] = weights(q[a:e, h], k, see, scale)
            o[a:e, h] = p @ v
    return o, lse


def _channels(D, rot, interleaved):
    """First and second channel of every rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(pos, freq):
    """pos * freq modulo a turn, with the product exact (11 more bits than fp64)."""
    a = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(freq, dtype=np.longdouble)[None]
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    return np.asarray(a - np.rint(a / turn) * turn, dtype=np.float64)


def rotate(x, pos, freq, interleaved=False, back=False):
    """x [N, h, D] with every pair turned by its token's angle (or back)."""
    y = x.copy()
    if freq is None or len(freq) == 0:
        return y
    t = angles(pos, freq)[:, None]
    c, s = np.cos(t), np.sin(t) * (-1 if back else 1)
    a, b = _channels(x.shape[-1], 2 * len(freq), interleaved)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_rope(x, w, pos, freq, eps=1e-6, interleaved=False):
    """One of q and k: x [N, h, D]. Rows of a negative position are 0."""
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    live = (np.asarray(pos) >= 0)[:, None, None]
    return np.where(live, rotate(x * r * (1.0 if w is None else w), pos, freq, interleaved), 0.0)


def norm_rope_backward(x, dy, w, pos, freq, eps=1e-6, interleaved=False):
    """(dx, dw) of sum(norm_rope(x) * dy)."""
    w = np.ones(x.shape[-1]) if w is None else w
    live = (np.asarray(pos) >= 0)[:, None, None]
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    z = x * r
    du = rotate(dy, pos, freq, interleaved, back=True)
    dx = r * (w * du - z * (w * du * z).mean(-1, keepdims=True))
    return np.where(live, dx, 0.0), np.where(live, du * z, 0.0).sum((0, 1))
