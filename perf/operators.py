"""What is timed of the packed token mixers: causal softmax attention with
grouped heads and linear attention with one decay per head, both over packed
documents (prompts and training steps), and the single-token steps of the two
recurrences.

``run`` computes a case with elementary torch operations in fp32 (``own`` is
false) or with this framework's kernels (``own`` is true); ``exact`` computes
it from the definitions in fp64.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SCORES = 1 << 28   # score elements the plain attention holds at once


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a packed training micro-batch's forward pass through a softmax layer
        # (8 rows of 8192 tokens of long documents, 4 query heads per kv head)
        dict(name="attn_flat_microbatch", op="attn", train=False, dtype="bf16", tokens=65536, tail=0, docs="lognormal",
             median=1500, doc_seed=2, max_segs=256, H=32, Hkv=8, D=128),
        # one short prompt: the call's latency
        dict(name="attn_short_prompt", op="attn", train=False, dtype="bf16", tokens=77, tail=0, docs="one", median=0,
             doc_seed=0, max_segs=1, H=16, Hkv=4, D=128),
        # a training step's forward and reverse pass on one packed sample
        dict(name="attn_train_sample", op="attn", train=True, dtype="bf16", tokens=8192, tail=0, docs="lognormal",
             median=800, doc_seed=1, max_segs=128, H=16, Hkv=4, D=128),
        # the same on many short documents with padding behind them, every head its own
        dict(name="attn_train_short_docs", op="attn", train=True, dtype="bf16", tokens=32768, tail=1640, docs="uniform",
             median=104, doc_seed=3, max_segs=1024, H=32, Hkv=32, D=64),
        # the small fp32 batch that models are debugged on
        dict(name="attn_train_tiny_f32", op="attn", train=True, dtype="f32", tokens=512, tail=20, docs="uniform",
             median=56, doc_seed=0, max_segs=16, H=4, Hkv=2, D=32),
        # the micro-batch's forward pass through a linear-attention layer
        dict(name="linear_flat_microbatch", op="linear", train=False, dtype="bf16", tokens=65536, tail=0,
             docs="lognormal", median=1500, doc_seed=2, max_segs=256, H=32, D=128, states=False),
        # a long prompt resumed from a state, its final state kept for decoding
        dict(name="linear_long_prompt", op="linear", train=False, dtype="bf16", tokens=32768, tail=0, docs="one",
             median=0, doc_seed=0, max_segs=1, H=16, D=128, states=True),
        # forward and reverse pass on one packed sample
        dict(name="linear_train_sample", op="linear", train=True, dtype="bf16", tokens=8192, tail=0,
             docs="lognormal", median=800, doc_seed=1, max_segs=128, H=16, D=128, states=False),
        # forward and reverse pass on many short documents
        dict(name="linear_train_short_docs", op="linear", train=True, dtype="bf16", tokens=32768, tail=1640,
             docs="uniform", median=104, doc_seed=3, max_segs=1024, H=32, D=64, states=False),
        # one request decoding: the step's latency
        dict(name="linear_step_one", op="linear_step", dtype="bf16", rows=1, idle=0, slots=4, H=16, D=128),
        # a full decoding batch, a few of its rows idle
        dict(name="linear_step_batch", op="linear_step", dtype="bf16", rows=128, idle=5, slots=160, H=32, D=128),
        # a decoding batch of the per-channel recurrence
        dict(name="kda_step_batch", op="kda_step", dtype="bf16", rows=48, idle=0, slots=64, H=32, D=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "linear", "linear", "linear", "linear_step", "kda_step"])
    f32 = rng.random() < 0.15
    if op in ("linear_step", "kda_step"):
        rows = _log_int(rng, 1, 128)
        return dict(op=op, dtype="f32" if f32 else "bf16", rows=rows, idle=rng.randint(0, rows // 8),
                    slots=rows + rng.randint(0, 32), H=rng.choice([4, 8, 16, 24, 32]), D=rng.choice([64, 128]))
    train = rng.random() < 0.5
    docs = rng.choice(["lognormal", "uniform", "one"])
    if f32:
        tokens, D = _log_int(rng, 48, 1024), rng.choice([32, 64])
        docs = rng.choice(["uniform", "one"])
    else:
        tokens, D = _log_int(rng, 33, 16384 if train else 32768), rng.choice([64, 128])
    if docs == "one":
        tokens = min(tokens, 16384)
    median = {"lognormal": rng.randint(200, 2000), "uniform": rng.randint(30, 300), "one": 0}[docs]
    tail = 0 if docs == "one" else rng.choice([0, rng.randint(0, tokens // 8)])
    Hkv = rng.choice([1, 2, 3, 4] if f32 else [1, 2, 4, 8])
    case = dict(op=op, train=train, dtype="f32" if f32 else "bf16", tokens=tokens, tail=tail, docs=docs,
                median=median, doc_seed=rng.randint(1, 1 << 20), max_segs=0, H=Hkv * rng.choice([1, 2, 4]), D=D)
    if op == "attn":
        case["Hkv"] = Hkv
    else:
        case["states"] = rng.random() < 0.5
    case["max_segs"] = len(_lengths(case)) + rng.randint(0, 9)
    return case


def _lengths(case):
    """Document lengths of a case (they fill tokens - tail)."""
    room = case["tokens"] - case["tail"]
    if case["docs"] == "one":
        return [room]
    rng = random.Random(case["doc_seed"])
    out = []
    while room > 0:
        if case["docs"] == "lognormal":
            n = int(round(case["median"] * math.exp(rng.gauss(0.0, 1.0))))
            n = min(max(n, 32), 8192)
        else:
            n = rng.randint(max(1, case["median"] // 13), 2 * case["median"])
        out.append(min(n, room))
        room -= out[-1]
    return out


# ---------------------------------------------------------------- the inputs

def _normal(gen, shape, dtype, unit=False):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if unit:
        x = x / x.square().sum(-1, keepdim=True).sqrt()
    return x.to(dtype)


def _log_decays(H):
    """One log decay per head, from heads that forget in a few tokens to heads
    that remember hundreds."""
    return torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], dtype=torch.float32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    op, H, D = case["op"], case["H"], case["D"]
    st = dict(case=case)
    if op in ("linear_step", "kda_step"):
        R, S = case["rows"], case["slots"]
        st["q"] = _normal(gen, (R, H, D), dt, unit=True)
        st["k"] = _normal(gen, (R, H, D), dt, unit=True)
        st["v"] = _normal(gen, (R, H, D), dt)
        slots = np.random.default_rng(seed).permutation(S)[:R].astype(np.int32)
        slots[R - case["idle"]:] = -1
        st["slots"] = torch.from_numpy(slots).cuda()
        st["state"] = _normal(gen, (S, H, D, D), torch.float32)
        if op == "linear_step":
            st["g"] = _log_decays(H)
        else:
            st["g"] = (-0.001 - 0.199 * torch.rand((R, H, D), generator=gen, device="cuda")).to(dt)
            st["beta"] = torch.rand((R, H), generator=gen, device="cuda").to(dt)
        return st
    lens = _lengths(case)
    N = case["tokens"]
    cu = np.full(case["max_segs"] + 1, sum(lens), dtype=np.int32)
    cu[:len(lens) + 1] = np.concatenate([[0], np.cumsum(lens)])
    st["lens"] = lens
    st["cu"] = torch.from_numpy(cu).cuda()
    if op == "attn":
        st["q"] = _normal(gen, (1, N, H, D), dt)
        st["k"] = _normal(gen, (1, N, case["Hkv"], D), dt)
        st["v"] = _normal(gen, (1, N, case["Hkv"], D), dt)
    else:
        st["q"] = _normal(gen, (1, N, H, D), dt, unit=True)
        st["k"] = _normal(gen, (1, N, H, D), dt, unit=True)
        st["v"] = _normal(gen, (1, N, H, D), dt)
        st["g"] = _log_decays(H)
        st["S0"] = _normal(gen, (case["max_segs"], H, D, D), torch.float32) if case["states"] else None
        st["dF"] = _normal(gen, (case["max_segs"], H, D, D), torch.float32) \
            if case["states"] and case["train"] else None
    if case["train"]:
        st["do"] = _normal(gen, (1, N, H, D), dt)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_attn(st):
    import packed_varlen_gated_amd as pkv
    train = st["case"]["train"]
    o, lse = pkv.attn_varlen(st["q"], st["k"], st["v"], st["cu"], output_lse=train)
    if not train:
        return {"o": o}
    gr = pkv.attn_varlen_backward(st["q"], st["k"], st["v"], o, lse, st["do"], st["cu"])
    return {"o": o, "dq": gr.dq, "dk": gr.dk, "dv": gr.dv}


def _own_linear(st):
    import packed_varlen_gated_amd as pkv
    case = st["case"]
    o, fs = pkv.chunk_linear_attn_varlen(st["q"], st["k"], st["v"], st["g"], st["cu"], initial_state=st["S0"],
                                         output_final_state=case["states"])
    out = {"o": o}
    if case["states"]:
        out["final_state"] = fs
    if case["train"]:
        gr = pkv.chunk_linear_attn_varlen_backward(st["q"], st["k"], st["v"], st["g"], st["do"], st["cu"],
                                                   initial_state=st["S0"], dfinal_state=st["dF"])
        out.update(dq=gr.dq, dk=gr.dk, dv=gr.dv)
        if case["states"]:
            out["d_initial_state"] = gr.d_initial_state
    return out


def _own_linear_step(st):
    import packed_varlen_gated_amd as pkv
    o = pkv.linear_attn_step(st["q"], st["k"], st["v"], st["g"], st["state"], st["slots"])
    return {"o": o, "state": st["state"]}


def _own_kda_step(st):
    import packed_varlen_gated_amd as pkv
    o = pkv.kda_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["slots"])
    return {"o": o, "state": st["state"]}


_OWN = {"attn": _own_attn, "linear": _own_linear, "linear_step": _own_linear_step, "kda_step": _own_kda_step}


# Plain forms. Documents of similar length are padded to one batch.

def _batches(lens, heads, quadratic):
    """Groups of documents as (start and length lists, padded length)."""
    starts = np.concatenate([[0], np.cumsum(lens)])
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    i = 0
    while i < len(order):
        L = lens[order[i]]
        per = heads * L * (L if quadratic else 128)
        n = max(1, min(len(order) - i, _SCORES // max(per, 1)))
        grp = [order[j] for j in range(i, i + n) if lens[order[j]] * 2 >= L]
        i += len(grp)
        yield grp, [int(starts[j]) for j in grp], [lens[j] for j in grp], L


def _index(starts, lens, L):
    """Token index [G, L] of padded documents, and which entries are real."""
    t = torch.arange(L)[None, :]
    s = torch.tensor(starts)[:, None]
    n = torch.tensor(lens)[:, None]
    return (s + torch.minimum(t, n - 1)).cuda(), (t < n).cuda()


def _gather(x, idx, real):
    """[N, h, d] -> fp32 [G, h, L, d], zeros where not real."""
    return (x[idx].float() * real[:, :, None, None]).transpose(1, 2)


def _scatter(out, y, idx, real):
    out[idx[real]] = y.transpose(1, 2)[real].to(out.dtype)


def _plain_attn(st):
    case = st["case"]
    H, Hkv, D, train = case["H"], case["Hkv"], case["D"], case["train"]
    rep = H // Hkv
    scale = 1.0 / math.sqrt(D)
    q, k, v = st["q"][0], st["k"][0], st["v"][0]
    o = torch.zeros_like(q)
    if train:
        do = st["do"][0]
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for _, starts, lens, L in _batches(st["lens"], H, True):
        idx, real = _index(starts, lens, L)
        G = len(lens)
        causal = torch.ones(L, L, dtype=torch.bool, device="cuda").tril()
        Q, K, V = _gather(q, idx, real), _gather(k, idx, real), _gather(v, idx, real)
        step = max(1, min(Hkv, _SCORES // max(1, G * rep * L * L)))
        O = torch.empty_like(Q)
        if train:
            DO = _gather(do, idx, real)
            DQ, DK, DV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
        for a in range(0, Hkv, step):
            b = min(Hkv, a + step)
            hs = slice(a * rep, b * rep)
            Qh = Q[:, hs].reshape(G, b - a, rep * L, D)
            S = torch.matmul(Qh, K[:, a:b].transpose(-1, -2)).view(G, b - a, rep, L, L) * scale
            S = S.masked_fill(~causal, -math.inf)
            S = torch.exp(S - S.amax(-1, keepdim=True))
            P = S / S.sum(-1, keepdim=True)
            Oh = torch.matmul(P.view(G, b - a, rep * L, L), V[:, a:b])
            O[:, hs] = Oh.view(G, (b - a) * rep, L, D)
            if not train:
                continue
            DOh = DO[:, hs].reshape(G, b - a, rep * L, D)
            DV[:, a:b] = torch.matmul(P.view(G, b - a, rep * L, L).transpose(-1, -2), DOh)
            DP = torch.matmul(DOh, V[:, a:b].transpose(-1, -2)).view(G, b - a, rep, L, L)
            delta = (DOh * Oh).sum(-1).view(G, b - a, rep, L, 1)
            DS = (P * (DP - delta)).view(G, b - a, rep * L, L)
            DQ[:, hs] = (torch.matmul(DS, K[:, a:b]) * scale).view(G, (b - a) * rep, L, D)
            DK[:, a:b] = torch.matmul(DS.transpose(-1, -2), Qh) * scale
        _scatter(o, O, idx, real)
        if train:
            _scatter(dq, DQ, idx, real)
            _scatter(dk, DK, idx, real)
            _scatter(dv, DV, idx, real)
    if not train:
        return {"o": o[None]}
    return {"o": o[None], "dq": dq[None], "dk": dk[None], "dv": dv[None]}


def _plain_chunks(q, k, v, g, S, lag):
    """out_t = sum_{s<=t} e^{g (t-s)} (q_t.k_s) v_s + e^{g (t+1-lag)} S^T q_t over
    64-token chunks; q, k [G, H, L, a], v [G, H, L, b], L a multiple of 64.
    Returns out and the states before every chunk and after the last."""
    G, H, L, a = q.shape
    C = 64
    n = L // C
    t = torch.arange(C, dtype=torch.float32, device="cuda")
    ex = lambda p: torch.exp(g[:, None] * p)
    rel = t[:, None] - t[None, :]
    M = torch.exp(g[:, None, None] * rel.clamp(min=0)) * (rel >= 0)
    qc, kc, vc = (x.reshape(G, H, n, C, x.shape[-1]) for x in (q, k, v))
    A = torch.matmul(qc, kc.transpose(-1, -2)) * M[None, :, None]
    out = torch.matmul(A, vc)
    add = torch.matmul((kc * ex(C - 1 - t + lag)[None, :, None, :, None]).transpose(-1, -2), vc)
    decay = torch.exp(g * C)[None, :, None, None]
    states = [S]
    for c in range(n):
        states.append(states[-1] * decay + add[:, :, c])
    before = torch.stack(states[:-1], 2)
    out = out + torch.matmul(qc * ex(t + 1 - lag)[None, :, None, :, None], before)
    return out.reshape(G, H, L, -1), states[-1]


def _plain_linear(st):
    case = st["case"]
    H, D, train, keep = case["H"], case["D"], case["train"], case["states"]
    q, k, v, g = st["q"][0], st["k"][0], st["v"][0], st["g"]
    o = torch.zeros_like(v)
    out = {"o": o[None]}
    slots = case["max_segs"]
    if keep:
        F = st["S0"].clone()                 # an empty slot keeps its state
        out["final_state"] = F
    if train:
        do = st["do"][0]
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        out.update(dq=dq[None], dk=dk[None], dv=dv[None])
        if keep:
            dI = st["dF"].clone()
            out["d_initial_state"] = dI
    for grp, starts, lens, L in _batches(st["lens"], H, False):
        L = (L + 63) // 64 * 64
        idx, real = _index(starts, lens, L)
        Q, K, V = _gather(q, idx, real), _gather(k, idx, real), _gather(v, idx, real)
        G = len(lens)
        zero = torch.zeros(G, H, D, D, device="cuda")
        S0 = st["S0"][grp] if keep else zero
        O, end = _plain_chunks(Q, K, V, g, S0, 0)
        _scatter(o, O, idx, real)
        behind = torch.tensor([L - n for n in lens], dtype=torch.float32).cuda()   # padded tokens only decay
        if keep:
            F[grp] = end * torch.exp(-g[None, :] * behind[:, None])[:, :, None, None]
        if not train:
            continue
        DO = _gather(do, idx, real)
        DQ, _ = _plain_chunks(DO, V, K, g, S0.transpose(-1, -2), 0)
        _scatter(dq, DQ, idx, real)
        # the adjoint walks the document backwards; reversed within its own length
        ridx = torch.tensor(lens).cuda()[:, None] - 1 - torch.arange(L, device="cuda")[None, :]
        ridx = ridx.clamp(min=0)[:, None, :, None]
        rev = lambda x: x.gather(2, ridx.expand(-1, x.shape[1], -1, x.shape[3])) * real[:, None, :, None]
        dF = st["dF"][grp] if keep else zero
        DV, end = _plain_chunks(rev(K), rev(Q), rev(DO), g, dF, 1)
        DK, _ = _plain_chunks(rev(V), rev(DO), rev(Q), g, dF.transpose(-1, -2), 1)
        _scatter(dv, rev(DV), idx, real)
        _scatter(dk, rev(DK), idx, real)
        if keep:
            dI[grp] = end * torch.exp(-g[None, :] * behind[:, None])[:, :, None, None]
    return out


def _plain_step(st, decay, beta):
    live = st["slots"] >= 0
    rows = st["slots"].clamp(min=0).long()
    S = st["state"][rows] * decay
    kv = st["k"].float()[..., :, None] * st["v"].float()[..., None, :]
    S = S + (kv if beta is None else kv * beta[..., None, None])
    o = (S * st["q"].float()[..., :, None]).sum(-2) * live[:, None, None]
    st["state"][rows[live]] = S[live]
    return {"o": o.to(st["v"].dtype), "state": st["state"]}


def _plain_linear_step(st):
    return _plain_step(st, torch.exp(st["g"])[None, :, None, None], None)


def _plain_kda_step(st):
    return _plain_step(st, torch.exp(st["g"].float())[..., None], st["beta"].float())


_PLAIN = {"attn": _plain_attn, "linear": _plain_linear, "linear_step": _plain_linear_step, "kda_step": _plain_kda_step}


# ---------------------------------------------------------------- the work

def work(case):
    """Every input read once, every output written once; the products of the
    definition (causal pairs of the softmax layer; update and readout of the
    recurrence)."""
    es = 2 if case["dtype"] == "bf16" else 4
    op, H, D = case["op"], case["H"], case["D"]
    if op in ("linear_step", "kda_step"):
        live = case["rows"] - case["idle"]
        small = live * H * D * es * (4 if op == "linear_step" else 5)
        return {"bytes": 2 * live * H * D * D * 4 + small, "flops": live * H * D * D * 4}
    lens = _lengths(case)
    real = sum(lens)
    if op == "attn":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        q, kv = real * H * D * es, real * case["Hkv"] * D * es
        if not case["train"]:
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * D * H * pairs}
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * D * H * pairs}
    x = real * H * D * es
    states = case["max_segs"] * H * D * D * 4 if case["states"] else 0
    if not case["train"]:
        return {"bytes": 4 * x + 2 * states, "flops": real * H * D * D * 4}
    return {"bytes": 8 * x + 4 * states, "flops": real * H * D * D * 14}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("linear_step", "kda_step"):
        return _exact_step(st)
    if len(st["lens"]) * case["H"] > 20000:   # head by head: over about 20 seconds
        return None
    return _exact_attn(st) if op == "attn" else _exact_linear(st)


def _exact_step(st):
    case = st["case"]
    q, k, v, state = (st[n].double() for n in ("q", "k", "v", "state"))
    o = torch.zeros_like(v)
    for r, s in enumerate(st["slots"].tolist()):
        if s < 0:
            continue
        if case["op"] == "linear_step":
            old = st["g"].double().exp()[:, None, None] * state[s]
            w = k[r]
        else:
            old = st["g"][r].double().exp()[:, :, None] * state[s]
            w = k[r] * st["beta"][r].double()[:, None]
        state[s] = old + w[:, :, None] * v[r][:, None, :]
        o[r] = torch.bmm(q[r][:, None, :], state[s])[:, 0]
    return {"o": o, "state": state}


def _exact_attn(st):
    """Softmax of each document's masked scores, head by head; the gradients by
    differentiating it."""
    case = st["case"]
    rep, D, train = case["H"] // case["Hkv"], case["D"], case["train"]
    full = {n: torch.zeros(st[s].shape, dtype=torch.float64, device="cuda")
            for n, s in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")) if train or n == "o"}
    a = 0
    for n in st["lens"]:
        mask = torch.full((n, n), -math.inf, dtype=torch.float64, device="cuda").triu(1)
        for h in range(case["Hkv"]):
            k = st["k"][0, a:a + n, h].double()
            v = st["v"][0, a:a + n, h].double()
            for j in range(h * rep, (h + 1) * rep):
                q = st["q"][0, a:a + n, j].double()
                leaves = [x.requires_grad_(train) for x in (q, k, v)]
                p = torch.softmax(q @ k.T / math.sqrt(D) + mask, -1)
                o = p @ v
                full["o"][0, a:a + n, j] = o.detach()
                if train:
                    d = torch.autograd.grad(o, leaves, st["do"][0, a:a + n, j].double())
                    full["dq"][0, a:a + n, j] = d[0]
                    full["dk"][0, a:a + n, h] += d[1]
                    full["dv"][0, a:a + n, h] += d[2]
        a += n
    return full


def _exact_linear(st):
    """The recurrence unrolled: every pair of a document's tokens weighted by
    e^{g (t - s)}, in blocks of rows; the gradients by differentiating it."""
    case = st["case"]
    H, train, keep = case["H"], case["train"], case["states"]
    zeros = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    out = {"o": zeros(st["v"])}
    if keep:
        out["final_state"] = st["S0"].double()
    if train:
        out.update(dq=zeros(st["q"]), dk=zeros(st["k"]), dv=zeros(st["v"]))
        if keep:
            out["d_initial_state"] = st["dF"].double()
    a = 0
    for i, n in enumerate(st["lens"]):
        t = torch.arange(n, dtype=torch.float64, device="cuda")
        for h in range(H):
            g = float(st["g"][h])
            q, k, v = (st[x][0, a:a + n, h].double().requires_grad_(train) for x in ("q", "k", "v"))
            S0 = st["S0"][i, h].double().requires_grad_(train) if keep else None
            rows = []
            for r in range(0, n, 4096):
                e = min(n, r + 4096)
                rel = t[r:e, None] - t[None, :e]
                w = torch.where(rel >= 0, torch.exp(g * rel.clamp(min=0)), 0.0)
                y = ((q[r:e] @ k[:e].T) * w) @ v[:e]
                if keep:
                    y = y + torch.exp(g * (t[r:e, None] + 1)) * (q[r:e] @ S0)
                rows.append(y)
            o = torch.cat(rows)
            out["o"][0, a:a + n, h] = o.detach()
            outs, cots = [o], []
            if keep:
                end = (k * torch.exp(g * (n - 1 - t))[:, None]).T @ v + math.exp(g * n) * S0
                out["final_state"][i, h] = end.detach()
                outs.append(end)
            if train:
                cots = [st["do"][0, a:a + n, h].double()] + ([st["dF"][i, h].double()] if keep else [])
                d = torch.autograd.grad(outs, [q, k, v] + ([S0] if keep else []), cots)
                for name, x in zip(("dq", "dk", "dv"), d):
                    out[name][0, a:a + n, h] = x
                if keep:
                    out["d_initial_state"][i, h] = d[3]
        a += n
    return out
