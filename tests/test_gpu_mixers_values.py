"""What single values of a call may and may not reach: rows of the softmax layer go by their own tokens alone, bit
by bit, and hold what the definition gives where values are not finite."""

import numpy as np
import pytest
import torch

import packed_varlen_gated_amd as pkv
from mixer_parity import E32, check, gamma, half_step, linear_bounds
from mixer_states import state_bound
from test_gpu_mixers import attn_case, attn_inputs, cu_gpu, host, lay, linear_case, linear_inputs, linear_run

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


def _with_special(ref, v, marks):
    """Rows of o where values of v are not finite (marks: token, kv head, channel, value): ref, the rows with those
    values finite, up to the first of them; from there on, since every weight of a token's own past is above 0, an
    infinity of the one sign that came, or NaN."""
    want = ref.clone()
    rep = ref.shape[2] // v.shape[2]
    for t, h, d, x in marks:
        want[0, t:, h * rep:(h + 1) * rep, d] += x      # inf + -inf, and anything + NaN, is NaN
    return want


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("s1,s2", [(70, 75), (70, 71), (64, 95), (3, 40), (40, 121), (500, 612), (1030, 1099), (0, 1)])
def test_attn_infinity_beside_a_later_value(dtype, D, s1, s2):
    """Row t attends to an infinity at s1 <= t and not to the value at s2 > t in its tile: it is that infinity."""
    N = 1100
    q, k, v, _ = attn_inputs(s1 + s2, N, 4, 2, D, dtype)
    for cu in forms(N):
        ref, rl = pkv.attn_varlen(q, k, v, cu)
        for x1, x2 in ((INF, NAN), (INF, INF), (-INF, INF), (-INF, -INF), (NAN, INF)):
            marks = [(s1, 0, 5, x1), (s2, 0, 5, x2), (s2, 1, 5, x1), (s1, 1, D - 1, x2), (s2, 0, 9, x2)]
            v2 = v.clone()
            for t, h, d, x in marks:
                v2[0, t, h, d] = x
            o, lse = pkv.attn_varlen(q, k, v2, cu)
            want = _with_special(ref, v, marks)
            same = (o == want) | (torch.isnan(o) & torch.isnan(want))
            assert same.all(), (x1, x2, cu is None, torch.nonzero(~same)[:4].tolist())
            assert torch.equal(lse, rl)


@pytest.mark.parametrize("dtype,Dk,Dv", [("f32", 32, 64), ("bf16", 32, 32), ("bf16", 64, 64), ("bf16", 128, 128),
                                         ("bf16", 64, 128), ("bf16", 128, 64)])
@pytest.mark.parametrize("states", [False, True])
def test_linear_results_do_not_go_by_what_else_is_asked_for(dtype, Dk, Dv, states):
    """The same o with and without the final state, the same gradients with and without the initial state's."""
    N, cu = lay([700, 0, 33, 900], 7)
    q, k, v, do, g, S0, dF = linear_inputs(7, N, 3, Dk, Dv, dtype, 4 if states else 0)
    c = cu_gpu(cu)
    a, fs = pkv.chunk_linear_attn_varlen(q, k, v, g, c, 0.5, initial_state=S0)
    b, none = pkv.chunk_linear_attn_varlen(q, k, v, g, c, 0.5, initial_state=S0, output_final_state=False)
    assert none is None and fs is not None and torch.equal(a, b)
    x, y = (pkv.chunk_linear_attn_varlen_backward(q, k, v, g, do, c, 0.5, initial_state=S0, dfinal_state=dF,
                                                  output_d_initial_state=w) for w in (True, False))
    assert y.d_initial_state is None
    for n in ("dq", "dk", "dv"):
        assert torch.equal(getattr(x, n), getattr(y, n)), n


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_linear_states_of_bf16_calls_are_fp32(Dk, Dv):
    lens, g = [31, 300, 0, 700, 90, 32], [-0.01, -0.05, -0.3]
    N, cu = lay(lens, 9)
    q, k, v, do, _, _, _ = linear_inputs(9, N, 3, Dk, Dv, "bf16")
    gd = torch.tensor(g, dtype=torch.float32, device=q.device)
    _, fs = pkv.chunk_linear_attn_varlen(q, k, v, gd, cu_gpu(cu), 0.3)
    gr = pkv.chunk_linear_attn_varlen_backward(q, k, v, gd, do, cu_gpu(cu), 0.3, output_d_initial_state=True)
    hq, hk, hv, hdo = (host(t)[0] for t in (q, k, v, do))
    gs = host(gd)
    for i, n in enumerate(lens):
        s = slice(int(cu[i]), int(cu[i]) + n)
        for h in range(3):
            w = np.exp(gs[h] * np.arange(n - 1, -1, -1))
            want = {"final": (hk[s, h] * w[:, None]).T @ hv[s, h],
                    "dinit": 0.3 * (hq[s, h] * np.exp(gs[h]) * w[::-1, None]).T @ hdo[s, h]}
            for name, got in (("final", fs), ("dinit", gr.d_initial_state)):
                x = host(got[i, h])
                rel = np.linalg.norm(x - want[name]) / max(np.linalg.norm(want[name]), 1e-30)
                assert rel <= state_bound(n, g[h]) if n else not x.any(), (name, n, g[h], rel)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32)])
def test_attn_off_the_bf16_matrix_path_long(dtype, D):
    attn_case([2100, 0, 300], 5, 2, 1, D, dtype, seed=D)
    attn_case([1999], 0, 2, 2, D, dtype, seed=D + 1, none=True)


@pytest.mark.parametrize("dtype,Dk,Dv", [("f32", 64, 64), ("f32", 32, 128), ("bf16", 32, 32), ("bf16", 128, 32)])
def test_linear_token_by_token_long(dtype, Dk, Dv):
    linear_case([2500, 0, 41], 6, 2, Dk, Dv, dtype, True, seed=Dk)


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("dtype,Dk,Dv", [("f32", 64, 64), ("bf16", 32, 64), ("bf16", 64, 64), ("bf16", 128, 128),
                                         ("bf16", 64, 128)])
def test_linear_growing_states(dtype, Dk, Dv, states):
    """Log decays above 0. A weight e^{g t} is off by 2 g t e for its argument, at most n e for g <= 0.5 and 2 n e for
    0.8: the bound's gamma(4 (n + Dk + Dv) + 64) allows for 4 n roundings where the sums have 3 n, and 4 (Dk + Dv) + 64
    more than n at these lengths.

    Element by element only. The normwise bound of mixer_parity.py takes a result for many independent roundings of
    like size; here 1 / (2 g) rows and, in each, 1 / (2 g) terms make the norm, one of each at g = 0.8, and a row with
    one term s is (a_t.b_s) w rounded once times c_s, rounded again: off by up to 2^-8 as a whole and 2^-8 per element,
    where the normwise bound allows for sqrt(3) times 2^-8 / sqrt(3). The element-wise bound has just these two."""
    for lens, tail, g, scale in (([70, 33, 0, 64], 3, [0.01, 0.2, 0.8], 0.5), ([700, 5], 0, [0.02, 0.05], 1.0)):
        N, cu = lay(lens, tail)
        H, end = len(g), int(cu[-1])
        q, k, v, do, _, S0, dF = linear_inputs(0, N, H, Dk, Dv, dtype, len(lens) if states else 0)
        gd = torch.tensor(g, dtype=torch.float32, device=q.device)
        got = linear_run(q, k, v, do, gd, S0, dF, cu_gpu(cu), scale)
        want = linear_bounds(host(q)[0], host(k)[0], host(v)[0], host(gd), host(do)[0], cu, scale, host(S0), host(dF),
                             dtype)
        for name, (ref, bound) in want.items():
            x = host(got[name])
            if name not in ("final", "dinit"):
                assert not x[0, end:].any(), name
                x = x[0]
            check(x, ref, bound, "f32", name)      # (no normwise bound)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("e", [60, 120, 125])
def test_linear_small_decay_weights(dtype, D, e):
    """A decay weight of 2^-e still counts: one token's large value, read by the next. The value 2^120 is exact, the
    weight is off by 4 e32 for exp and 2 e32 of its argument (e ln 2 < 87: 174 e32), o by its rounding besides."""
    q, k, v, _ = (torch.zeros_like(t) for t in attn_inputs(0, 2, 1, 1, D, dtype))
    k[0, 0, 0, 0] = 1.0
    q[0, 1, 0, 0] = 1.0
    v[0, 0, 0, 3] = 2.0 ** 120
    g = torch.tensor([-e * np.log(2)], dtype=torch.float32, device=q.device)
    o, fs = pkv.chunk_linear_attn_varlen(q, k, v, g)
    want = 2.0 ** 120 * np.exp(float(g[0]))
    rel = gamma(180)
    assert abs(float(fs[0, 0, 0, 3]) - want) <= rel * want
    assert abs(float(o[0, 1, 0, 3]) - want) <= (rel + 2.01 * half_step(dtype)) * want


@pytest.mark.parametrize("Hkv", [65536, 4096])
def test_attn_most_heads(Hkv):
    """65536 heads of 128: rows 16 MiB apart, so a tile of 128 spans almost 2^31 bytes. A few heads equal a call of
    their own with as many per kv head; dk and dv as one of two sum orders (test_offsets_past_32_bits)."""
    H, N, D, rep = 65536, 130, 128, 65536 // Hkv
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.empty(1, N, h, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
                   for h in (H, Hkv, Hkv, H))
    o, lse = pkv.attn_varlen(q, k, v)
    gr = pkv.attn_varlen_backward(q, k, v, o, lse, do)
    for a in (0, 777 % Hkv, Hkv - 1):
        hs = slice(a * rep, (a + 1) * rep)
        q1, do1 = (t[:, :, hs].contiguous() for t in (q, do))
        k1, v1 = (t[:, :, a:a + 1].contiguous() for t in (k, v))
        o1, lse1 = pkv.attn_varlen(q1, k1, v1)
        gr1 = pkv.attn_varlen_backward(q1, k1, v1, o1, lse1, do1)
        assert torch.equal(o[:, :, hs], o1) and torch.equal(lse[hs], lse1) and torch.equal(gr.dq[:, :, hs], gr1.dq)
        hq, hdo = (t[0].double().transpose(0, 1) for t in (q1, do1))
        hk, hv = k1[0, :, 0].double(), v1[0, :, 0].double()
        P = torch.softmax((hq @ hk.T / D ** 0.5).masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -INF), -1)
        dP = hdo @ hv.T
        dS = (P * (dP - (P * dP).sum(-1, keepdim=True))).abs() / D ** 0.5
        for name, t in (("dk", (dS.transpose(1, 2) @ hq.abs()).sum(0)), ("dv", (P.transpose(1, 2) @ hdo.abs()).sum(0))):
            x, y = getattr(gr, name)[0, :, a].double(), getattr(gr1, name)[0, :, 0].double()
            # (1.02: P and dS are bf16 there)
            bound = 2.0 ** -7 * torch.maximum(x.abs(), y.abs()) + 2 * gamma(rep * N) * 1.02 * t
            assert ((x - y).abs() <= bound).all(), (name, a)


def test_linear_most_heads():
    H, N, D = 65536, 130, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, do = (torch.empty(1, N, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4))
    g = torch.linspace(-2, 0, H, device="cuda")
    cu = cu_gpu([0, 67, 67, 129])
    S0 = torch.empty(3, H, D, D, device="cuda").normal_(generator=gen)
    o, fs = pkv.chunk_linear_attn_varlen(q, k, v, g, cu, initial_state=S0)
    gr = pkv.chunk_linear_attn_varlen_backward(q, k, v, g, do, cu, initial_state=S0, dfinal_state=S0)
    hs = torch.tensor([0, 777, H - 1], device="cuda")
    one = [t[:, :, hs].contiguous() for t in (q, k, v, do)]
    o1, fs1 = pkv.chunk_linear_attn_varlen(*one[:3], g[hs], cu, initial_state=S0[:, hs].contiguous())
    gr1 = pkv.chunk_linear_attn_varlen_backward(*one[:3], g[hs], one[3], cu, initial_state=S0[:, hs].contiguous(),
                                                dfinal_state=S0[:, hs].contiguous())
    assert torch.equal(o[:, :, hs], o1) and torch.equal(fs[:, hs], fs1)
    for a, b in zip(gr[:3], gr1[:3]):
        assert torch.equal(a[:, :, hs], b)
    assert torch.equal(gr.d_initial_state[:, hs], gr1.d_initial_state)


def _dq_bound(q, k, v, do, n, scale, u):
    """dq of a segment's first n tokens, and the error it may have where delta = sum_s P_ts dP_ts is formed in fp32
    (not from o, whose rounding is as large as what is left of a row that has few keys; the first row's dq is 0).
    Weights as in mixer_parity.attn_bounds: a factor within exp(s_err + the error of lse + 8 e), lse within 2 s_err and
    the sum's gamma_n; dP and delta are fp32 sums, dS is rounded once on its way into the product, dq once."""
    Q, K, V, DO = (x[:n] for x in (q, k, v, do))
    D = Q.shape[1]
    mask = np.tril(np.ones((n, n), dtype=bool))
    s = scale * (Q @ K.T)
    top = np.where(mask, s, -np.inf).max(axis=1, keepdims=True)
    P = np.where(mask, np.exp(s - top), 0)
    P /= P.sum(1, keepdims=True)
    s_err = gamma(D + 2) * abs(scale) * (abs(Q) @ abs(K).T) + 2 * E32 * abs(s)
    s_top = np.where(mask, s_err, 0).max(axis=1, keepdims=True)
    l_err = np.expm1(2 * s_top + 8 * E32) + gamma(n + 4)
    lse_err = 2 * l_err + s_top + 8 * E32 * (1 + 2 * abs(s).max(axis=1, keepdims=True) + np.log(n))
    p_err = np.expm1(s_err + lse_err + 8 * E32)
    dP = DO @ V.T
    p_abs = gamma(D + 2) * (abs(DO) @ abs(V).T)                                    # of dP
    delta = (P * dP).sum(1, keepdims=True)
    d_err = (P * ((p_err + gamma(n + 4)) * abs(dP) + (1 + p_err) * p_abs)).sum(1, keepdims=True)
    dS = P * (dP - delta)
    ds_err = P * (1 + p_err) * ((d_err + p_abs) * (1 + u) + (p_err + u + 2 * E32) * abs(dP - delta))
    dq = scale * dS @ K
    b = abs(scale) * (ds_err @ abs(K) + gamma(n + 8) * (abs(dS) @ abs(K)))
    return dq, b + u * (abs(dq) + b) + 1e-37


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("none", [False, True])
def test_attn_dq_of_a_segments_first_tokens(D, none):
    lens = [300] if none else [1, 2, 5, 0, 17, 31, 32, 33, 64, 300]
    N, cu = lay(lens, 0 if none else 6)
    q, k, v, do = attn_inputs(D, N, 4, 2, D, "bf16")
    c = None if none else cu_gpu(cu)
    o, lse = pkv.attn_varlen(q, k, v, c)
    gr = pkv.attn_varlen_backward(q, k, v, o, lse, do, c)
    hq, hk, hv, hdo, got = (host(t)[0] for t in (q, k, v, do, gr.dq))
    for i, n in enumerate(lens):
        a, m = int(cu[i]), min(n, 32)
        for h in range(4 if m else 0):
            ref, bound = _dq_bound(hq[a:, h], hk[a:, h // 2], hv[a:, h // 2], hdo[a:, h], m, D ** -0.5, half_step("bf16"))
            err = abs(got[a:a + m, h] - ref)
            assert (err <= bound).all(), (n, h, float((err / bound).max()), int((err / bound).argmax()) // D)
