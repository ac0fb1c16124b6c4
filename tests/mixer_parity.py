"""Error bounds of the mixers' kernels against their fp64 oracle.

Every bound is element-wise and follows the arithmetic, with u = half a step of
the tensors' type (2^-8 for bf16, 2^-24 for fp32), e = 2^-24 and
gamma_n = n e / (1 - n e) for fp32 sums of n terms in any order (Higham,
Accuracy and Stability of Numerical Algorithms, section 3.1). exp and log of the
device are within 4 e relative. For bf16 a second, normwise bound holds: a
rounding's relative error is at most 2^-8 and, over many values, spread over
that interval, so its root mean square is at most 2^-8 / sqrt(3); at most three
roundings meet in a result (one on the way into each of two products, one of
the output), independent: sqrt(3) 2^-8 / sqrt(3) = 2^-8 = 3.9e-3.
"""

import numpy as np

from oracle import mixers

E32 = 2.0 ** -24
RELL2_BF16 = 2.0 ** -8


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else E32


def gamma(n):
    return n * E32 / (1 - n * E32)


def check(got, ref, bound, dtype, what, extra=0.0):
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    over = err > bound
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.size} outside, worst "
                            f"{float((err / np.maximum(bound, 1e-300)).max()):.3g} of the bound")
    n = np.linalg.norm(ref)
    if dtype == "bf16" and n > 0 and ref.size >= 2000:
        rel, top = float(np.linalg.norm(err) / n), float(np.hypot(RELL2_BF16, extra / n))
        assert rel <= top, f"{what}: rel-L2 {rel:.3e} > {top:.3e}"


def attn_bounds(q, k, v, do, cu, scale, dtype):
    """Oracle results and element-wise bounds of the softmax calls:
    {name: (reference, bound, norm of delta's part)} for o, lse, dq, dk, dv.

    A score's error is at most s_err = gamma_{D+2} scale |q|.|k| + 2 e |s| (fp32
    product sums, the factor of exp2's argument), the same bound holds for the
    running maximum that is subtracted, so a weight is off by a factor within
    exp(+-(2 s_err + 8 e)); weights are rounded to the tensors' type before the
    second product (bf16 kernels), and the row's sum carries the same relative
    error as the weights.
    """
    u = half_step(dtype)
    N, Hq, D = q.shape
    rep = Hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    o, lse = mixers.attn_varlen(q, k, v, cu, scale)
    dq, dk, dv = mixers.attn_varlen_backward(q, k, v, do, cu, scale)
    b = {"o": np.zeros_like(q), "lse": np.zeros_like(lse), "dq": np.zeros_like(q), "dk": np.zeros_like(k),
         "dv": np.zeros_like(v)}
    part = {"dq": np.zeros_like(q), "dk": np.zeros_like(k)}   # squared
    for a, e in [(0, N)] if cu is None else list(zip(cu[:-1], cu[1:])):
        n = int(e - a)
        if n == 0:
            continue
        mask = np.tril(np.ones((n, n), dtype=bool))
        for h in range(Hq):
            g = h // rep
            Q, K, V, DO = q[a:e, h], k[a:e, g], v[a:e, g], do[a:e, h]
            s = np.where(mask, scale * (Q @ K.T), 0)
            s_err = np.where(mask, gamma(D + 2) * abs(scale) * (abs(Q) @ abs(K).T) + 2 * E32 * abs(s), 0)
            top = s_err.max(axis=1, keepdims=True)
            w_err = np.expm1(s_err + top + 8 * E32)             # of a weight, relative
            l_err = w_err.max(axis=1, keepdims=True) + gamma(n + 4)  # of the row's sum, relative
            P = np.where(mask, np.exp(s - lse[h, a:e][:, None]), 0)
            rel = (1 + w_err) * (1 + u) * (1 + 2 * l_err) - 1 + gamma(n + 8)
            b["o"][a:e, h] = (P * rel) @ abs(V) + u * abs(o[a:e, h])
            b["lse"][h, a:e] = (2 * l_err + top)[:, 0] + 8 * E32 * (1 + abs(lse[h, a:e]) + abs(s).max(axis=1))
            # reverse pass: P from lse, o rounded once on its way into delta
            p_err = np.expm1(s_err + b["lse"][h, a:e][:, None] + 8 * E32)
            dP = DO @ V.T
            delta = (DO * o[a:e, h]).sum(1, keepdims=True)
            aO = abs(DO) @ abs(V).T
            d_err = gamma(D + 4) * (aO + (abs(DO) * abs(o[a:e, h])).sum(1, keepdims=True)) + \
                (abs(DO) * b["o"][a:e, h]).sum(1, keepdims=True)
            dS = P * (dP - delta)
            ds_err = P * (1 + p_err) * (d_err * (1 + u) + (p_err + u) * abs(dP - delta))
            b["dq"][a:e, h] = abs(scale) * (ds_err @ abs(K) + gamma(n + 8) * (abs(dS) @ abs(K)))
            b["dk"][a:e, g] += abs(scale) * (ds_err.T @ abs(Q) + gamma(rep * n + 8) * (abs(dS).T @ abs(Q)))
            b["dv"][a:e, g] += (P * (p_err + u * (1 + p_err) + gamma(rep * n + 8))).T @ abs(DO)
            r = 2.0 ** -8 / np.sqrt(3) * np.sqrt(((DO * o[a:e, h]) ** 2).sum(1, keepdims=True))
            part["dq"][a:e, h] = (scale * r * (P @ K)) ** 2
            part["dk"][a:e, g] += scale ** 2 * ((P ** 2).T @ (r * Q) ** 2)
    for name, ref in (("dq", dq), ("dk", dk), ("dv", dv)):
        b[name] += u * (abs(ref) + b[name])
    refs = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    return {x: (refs[x], b[x] + 1e-37, float(np.sqrt(part[x].sum())) if x in part else 0.0) for x in refs}


def linear_bounds(q, k, v, g, do, cu, scale, S0, dF, dtype):
    """The same for the linear-attention calls (o, final, dq, dk, dv, dinit).

    A result is a sum of products; the sum of the products' absolute values is
    the oracle run on absolute values (the decays are positive). Each product
    passes one rounding of its weight or of the state to the tensors' type, a
    split of the decayed key into bf16 parts whose remainder is at most 2^-16,
    and fp32 sums over at most n tokens; a decay e^{g t} carries
    t (|g| e + ...) from its argument, (8 + 2 |g| t) e; a term that far back is
    weighted by e^{g t}, and x e^{-x} < 0.4: 16 e covers it for any t. States
    see no rounding of the weight. The output is rounded once.
    """
    u = half_step(dtype)
    n = int(max(np.diff(cu))) if cu is not None else q.shape[0]
    split = 2.0 ** -16 if dtype == "bf16" else 0.0
    f = gamma(4 * (n + q.shape[2] + v.shape[2]) + 64) + 16 * E32 + split
    A = lambda x: None if x is None else np.abs(x)
    o, fs = mixers.linear_attn_varlen(q, k, v, g, cu, scale, S0)
    ao, afs = mixers.linear_attn_varlen(A(q), A(k), A(v), g, cu, abs(scale), A(S0))
    dq, dk, dv, di = mixers.linear_attn_varlen_backward(q, k, v, g, do, cu, scale, S0, dF)
    adq, adk, adv, adi = mixers.linear_attn_varlen_backward(A(q), A(k), A(v), g, A(do), cu, abs(scale), A(S0), A(dF))
    out = {}
    for name, ref, top in (("o", o, ao), ("dq", dq, adq), ("dk", dk, adk), ("dv", dv, adv)):
        out[name] = (ref, (u * (1 + u) + f) * top + u * abs(ref) + 1e-37)
    for name, ref, top in (("final", fs, afs), ("dinit", di, adi)):
        out[name] = (ref, f * top + 1e-37)
    return out
