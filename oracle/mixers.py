"""fp64 oracle of the packed token mixers next to KDA and of the single-token steps.

``attn_varlen``: causal softmax attention inside each segment ("Drill: Sequence
Packing from scratch", The math: a token sees the earlier tokens of its own
document), grouped heads. ``linear_attn_varlen``: the recurrence of RFC-0026
Background with one decay per head in place of the gate per channel and no
beta, token by token. The reverse passes walk the chain rule of these forms.
The steps are the recurrences' one-token case.

Pinned (tests/test_oracle_mixers.py): brute force over pairs in plain Python,
closed forms (one key, equal scores, geometric series, zero decay), KDA with a
broadcast gate, central finite differences of every gradient.
"""

import numpy as np


def _segments(cu, N):
    if cu is None:
        return [(0, 0, N)]
    return [(i, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def _probs(q, k, scale):
    s = scale * (q @ k.T)
    s = np.where(np.tril(np.ones(s.shape, dtype=bool)), s, -np.inf)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    z = p.sum(axis=1, keepdims=True)
    return p / z, (m + np.log(z))[:, 0]


def attn_varlen(q, k, v, cu=None, scale=None):
    """q [N, Hq, D], k and v [N, Hkv, D] -> (o [N, Hq, D], lse [Hq, N])."""
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    o = np.zeros((N, Hq, D))
    lse = np.full((Hq, N), -np.inf)
    for _, a, e in _segments(cu, N):
        if e > a:
            for h in range(Hq):
                p, lse[h, a:e] = _probs(q[a:e, h], k[a:e, h // rep], scale)
                o[a:e, h] = p @ v[a:e, h // rep]
    return o, lse


def attn_varlen_backward(q, k, v, do, cu=None, scale=None):
    """(dq, dk, dv) of sum(o * do)."""
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for _, a, e in _segments(cu, N):
        if e > a:
            for h in range(Hq):
                g = h // rep
                p, _ = _probs(q[a:e, h], k[a:e, g], scale)
                dp = do[a:e, h] @ v[a:e, g].T
                ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
                dq[a:e, h] = scale * ds @ k[a:e, g]
                dk[a:e, g] += scale * ds.T @ q[a:e, h]
                dv[a:e, g] += p.T @ do[a:e, h]
    return dq, dk, dv


def linear_attn_varlen(q, k, v, g, cu=None, scale=1.0, initial_state=None):
    """q, k [N, H, Dk], v [N, H, Dv], g [H] -> (o [N, H, Dv], final [segs, H, Dk, Dv])."""
    N, H, Dk = q.shape
    Dv = v.shape[2]
    segs = _segments(cu, N)
    o = np.zeros((N, H, Dv))
    fs = np.zeros((len(segs), H, Dk, Dv))
    lam = np.exp(g)[:, None, None]
    for i, a, e in segs:
        S = np.zeros((H, Dk, Dv)) if initial_state is None else initial_state[i].astype(np.float64)
        for t in range(a, e):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hde,hd->he", S, q[t])
        fs[i] = S
    return o, fs


def linear_attn_varlen_backward(q, k, v, g, do, cu=None, scale=1.0, initial_state=None, dfinal=None):
    """(dq, dk, dv, d_initial) of sum(o * do) + sum(final * dfinal)."""
    N, H, Dk = q.shape
    Dv = v.shape[2]
    segs = _segments(cu, N)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    di = np.zeros((len(segs), H, Dk, Dv))
    lam = np.exp(g)[:, None, None]
    for i, a, e in segs:
        S = np.zeros((H, Dk, Dv)) if initial_state is None else initial_state[i].astype(np.float64)
        for t in range(a, e):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hde,he->hd", S, do[t])
        dS = np.zeros((H, Dk, Dv)) if dfinal is None else dfinal[i].astype(np.float64)
        for t in range(e - 1, a - 1, -1):
            dS = dS + scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = np.einsum("hde,he->hd", dS, v[t])
            dv[t] = np.einsum("hde,hd->he", dS, k[t])
            dS = lam * dS
        di[i] = dS
    return dq, dk, dv, di


def step(q, k, v, decay, weight, state, slots, scale=1.0):
    """One token of R requests: state [S, H, Dk, Dv] (a copy is updated), decay broadcastable to
    [R, H, Dk], weight to [R, H] (KDA's beta; 1 for linear attention). Returns (o, state)."""
    R, H, Dk = q.shape
    state = state.astype(np.float64).copy()
    o = np.zeros(v.shape)
    decay = np.broadcast_to(decay, (R, H, Dk))
    weight = np.broadcast_to(weight, (R, H))
    seen = set()
    for r in range(R):
        s = int(slots[r])
        if s < 0 or s >= state.shape[0] or s in seen:
            continue
        seen.add(s)
        state[s] = decay[r][:, :, None] * state[s] + (weight[r][:, None] * k[r])[:, :, None] * v[r][:, None, :]
        o[r] = scale * np.einsum("hde,hd->he", state[s], q[r])
    return o, state
