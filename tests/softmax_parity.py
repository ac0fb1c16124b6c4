"""Error bounds of the softmax layer's kernels against their fp64 oracle; the notation
and the derivations of mixer_parity.py (u half a step of the tensors' type, e = 2^-24,
gamma_n for fp32 sums of n terms), with the pairs that a window or a cache leaves."""

import numpy as np

from mixer_parity import E32, gamma, half_step
from oracle import softmax


def _row_bounds(Q, K, V, see, scale, dtype):
    """(P, o, lse, o's bound, lse's bound, scores' error) of one head; rows that see nothing have bounds of 0.

    As attn_bounds of mixer_parity.py; where a walk is cut into pieces that are joined, each piece's
    weights are scaled once more by an exponential of a difference of two maxima (within the
    2 s_err + 8 e that a weight has already, taken twice here) and summed once more (n + 64 terms).
    """
    D, n = Q.shape[1], K.shape[0]
    u = half_step(dtype)
    P, lse = softmax.weights(Q, K, see, scale)
    any_ = see.any(1)
    o = P @ V
    s = np.where(see, scale * (Q @ K.T), 0)
    s_err = np.where(see, gamma(D + 2) * abs(scale) * (abs(Q) @ abs(K).T) + 2 * E32 * abs(s), 0)
    top = s_err.max(axis=1, keepdims=True, initial=0)
    w_err = np.expm1(s_err + 3 * top + 16 * E32)
    l_err = w_err.max(axis=1, keepdims=True, initial=0) + gamma(n + 64)
    rel = (1 + w_err) * (1 + u) * (1 + 2 * l_err) - 1 + gamma(n + 64)
    b_o = (P * rel) @ abs(V) + u * abs(o)
    safe = np.where(any_, lse, 0)
    b_l = (2 * l_err + top)[:, 0] + 8 * E32 * (1 + abs(safe) + abs(s).max(axis=1, initial=0))
    return P, o, lse, b_o, np.where(any_, b_l, 0), s_err


def window_bounds(q, k, v, do, window, sinks, cu, scale, dtype):
    """{name: (reference, bound, norm of delta's part)} for o, lse, dq, dk, dv."""
    u = half_step(dtype)
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    dq, dk, dv = softmax.attn_window_varlen_backward(q, k, v, do, window, sinks, cu, scale)
    ref = dict(o=np.zeros_like(q), lse=np.full((Hq, N), -np.inf), dq=dq, dk=dk, dv=dv)
    b = {x: np.zeros_like(y) for x, y in ref.items()}
    part = {"dq": np.zeros_like(q), "dk": np.zeros_like(k)}   # squared
    for a, e in [(0, N)] if cu is None else list(zip(cu[:-1], cu[1:])):
        n = int(e - a)
        if n == 0:
            continue
        see = softmax.visible(np.arange(n), np.arange(n), window, sinks)
        for h in range(Hq):
            g = h // rep
            Q, K, V, DO = q[a:e, h], k[a:e, g], v[a:e, g], do[a:e, h]
            P, o, lse, b_o, b_l, s_err = _row_bounds(Q, K, V, see, scale, dtype)
            ref["o"][a:e, h], ref["lse"][h, a:e], b["o"][a:e, h], b["lse"][h, a:e] = o, lse, b_o, b_l
            p_err = np.expm1(s_err + b_l[:, None] + 8 * E32)
            dP = DO @ V.T
            delta = (DO * o).sum(1, keepdims=True)
            aO = abs(DO) @ abs(V).T
            d_err = gamma(D + 4) * (aO + (abs(DO) * abs(o)).sum(1, keepdims=True)) + \
                (abs(DO) * b_o).sum(1, keepdims=True)
            dS = P * (dP - delta)
            ds_err = P * (1 + p_err) * (d_err * (1 + u) + (p_err + u) * abs(dP - delta))
            b["dq"][a:e, h] = abs(scale) * (ds_err @ abs(K) + gamma(n + 8) * (abs(dS) @ abs(K)))
            b["dk"][a:e, g] += abs(scale) * (ds_err.T @ abs(Q) + gamma(rep * n + 64) * (abs(dS).T @ abs(Q)))
            b["dv"][a:e, g] += (P * (p_err + u * (1 + p_err) + gamma(rep * n + 64))).T @ abs(DO)
            r = 2.0 ** -8 / np.sqrt(3) * np.sqrt(((DO * o) ** 2).sum(1, keepdims=True))
            part["dq"][a:e, h] = (scale * r * (P @ K)) ** 2
            part["dk"][a:e, g] += scale ** 2 * ((P ** 2).T @ (r * Q) ** 2)
    for name in ("dq", "dk", "dv"):
        b[name] += u * (abs(ref[name]) + b[name])
    return {x: (ref[x], b[x] + 1e-37, float(np.sqrt(part[x].sum())) if x in part else 0.0) for x in ref}


def paged_bounds(q, k_pages, v_pages, table, lens, cu, window, sinks, scale, dtype):
    """{name: (reference, bound)} for o and lse."""
    N, Hq, D = q.shape
    size, Hkv = k_pages.shape[1:3]
    scale = 1 / np.sqrt(D) if scale is None else scale
    o, lse = np.zeros((N, Hq, D)), np.full((Hq, N), -np.inf)
    b_o, b_l = np.zeros_like(o), np.zeros((Hq, N))
    cu = np.arange(len(lens) + 1) if cu is None else cu
    for r in range(len(lens)):
        a, e, n = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if e == a or n == 0:
            continue
        at = softmax.places(table[r], n, size)
        see = softmax.visible(np.arange(n - (e - a), n), np.arange(n), window, sinks)
        for h in range(Hq):
            k, v = (x.reshape(-1, Hkv, D)[at, h // (Hq // Hkv)] for x in (k_pages, v_pages))
            _, o[a:e, h], lse[h, a:e], b_o[a:e, h], b_l[h, a:e], _ = _row_bounds(q[a:e, h], k, v, see, scale, dtype)
    return dict(o=(o, b_o + 1e-37), lse=(lse, b_l + 1e-37))


# sin and cos: the reduced angle is rounded to fp32 (half a turn at most: pi 2^-24) and the functions are
# within 4 e; before that it is a product of fp64 numbers, two of them rounded: 3 2^-53 of the whole angle.
def _turn_err(pos, freq):
    n = 0 if freq is None else len(freq)
    if n == 0:
        return 0.0
    far = np.abs(np.asarray(pos, dtype=np.float64))[:, None] * np.abs(np.asarray(freq, dtype=np.float64)).max()
    return 8 * E32 + (3 * 2.0 ** -53 * far)[:, :, None]


def _pair_sum(x, freq, interleaved):
    """|x| of both members of every pair, at both."""
    y = abs(x).copy()
    if freq is not None and len(freq):
        a, b = softmax._channels(x.shape[-1], 2 * len(freq), interleaved)
        y[..., a] = y[..., b] = abs(x[..., a]) + abs(x[..., b])
    return y


def norm_rope_bounds(x, dy, w, pos, freq, eps, interleaved, dtype):
    """(reference, bound) of y, dx and dw of one of q and k. fp32 throughout: the mean is a sum of D squares,
    the norm's factor and a product or two are rounded on the way (16 roundings cover them)."""
    u = half_step(dtype)
    D = x.shape[-1]
    live = (np.asarray(pos) >= 0)[:, None, None]
    w1 = np.ones(D) if w is None else w
    g = gamma(D + 32)
    turn = _turn_err(pos, freq) + gamma(4)
    y = softmax.norm_rope(x, w, pos, freq, eps, interleaved)
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    z = x * r
    b_y = _pair_sum(z * w1, freq, interleaved) * (g + turn) * (1 + u) + u * abs(y)
    dx, dw = softmax.norm_rope_backward(x, dy, w, pos, freq, eps, interleaved)
    du = np.where(live, softmax.rotate(dy, pos, freq, interleaved, back=True), 0)
    E = np.where(live, _pair_sum(dy, freq, interleaved) * turn, 0)
    mean = lambda t: t.mean(-1, keepdims=True)
    s = mean(w1 * du * z)
    s_err = mean(abs(w1) * E * abs(z)) + g * mean(abs(w1 * du * z))
    b_dx = r * (abs(w1) * E + abs(z) * s_err + g * (abs(w1 * du) + abs(z * s))) * (1 + u) + u * abs(dx)
    terms = abs(du * z).sum((0, 1))
    b_dw = (E * abs(z)).sum((0, 1)) * (1 + g) + (g + gamma(x.shape[0] * x.shape[1])) * terms
    tiny = 1e-37
    return dict(y=(y, np.where(live, b_y, 0) + tiny), dx=(dx, np.where(live, b_dx, 0) + tiny), dw=(dw, b_dw + tiny))
