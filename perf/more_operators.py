"""What is timed of the softmax layer around the packed causal attention: the norms
of queries and keys with the rotation by position, attention through a sliding
window with a few first tokens that stay visible, and, for serving, attention of
new tokens over a paged cache and the call that fills the cache.

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
_SCORES = 1 << 28   # score elements that are held at once
_EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the forward pass of a packed training micro-batch (8 rows of 8192 tokens of long documents): queries and
        # keys as they lie in the result of one projection for q, k and v
        dict(name="norm_rope_flat_microbatch", op="norm_rope", train=False, dtype="bf16", tokens=65536,
             docs="lognormal", median=1500, doc_seed=2, H=32, Hkv=8, D=128, rot=128, interleaved=False, fused=True,
             far=0),
        # forward and reverse pass on one packed sample, half of each head rotated
        dict(name="norm_rope_train_sample", op="norm_rope", train=True, dtype="bf16", tokens=8192, docs="lognormal",
             median=800, doc_seed=1, H=16, Hkv=4, D=128, rot=64, interleaved=False, fused=False, far=0),
        # the micro-batch's forward pass through a windowed layer
        dict(name="window_flat_microbatch", op="window", train=False, dtype="bf16", tokens=65536, tail=0,
             docs="lognormal", median=1500, doc_seed=2, max_segs=256, H=32, Hkv=8, D=128, window=1024, sinks=4),
        # a training step's forward and reverse pass on one packed sample
        dict(name="window_train_sample", op="window", train=True, dtype="bf16", tokens=8192, tail=0,
             docs="lognormal", median=800, doc_seed=1, max_segs=128, H=16, Hkv=4, D=128, window=512, sinks=0),
        # the same on one long document with visible first tokens, every head its own
        dict(name="window_train_long_doc", op="window", train=True, dtype="bf16", tokens=16384, tail=0, docs="one",
             median=0, doc_seed=0, max_segs=1, H=16, Hkv=16, D=64, window=256, sinks=4),
        # the small fp32 batch that models are debugged on
        dict(name="window_train_tiny_f32", op="window", train=True, dtype="f32", tokens=512, tail=20, docs="uniform",
             median=56, doc_seed=0, max_segs=16, H=4, Hkv=2, D=32, window=24, sinks=2),
        # a decoding batch of requests of mixed lengths, a few rows idle
        dict(name="paged_decode_batch", op="paged", dtype="bf16", requests=64, idle=3, new=1, chunks=0,
             context=2000, longest=16384, ctx_seed=1, H=32, Hkv=8, D=128, page=64, window=0, sinks=0),
        # one request with a long context
        dict(name="paged_decode_long", op="paged", dtype="bf16", requests=1, idle=0, new=1, chunks=0,
             context=131072, longest=131072, ctx_seed=0, H=32, Hkv=8, D=128, page=64, window=0, sinks=0),
        # a larger decoding batch of a windowed layer
        dict(name="paged_decode_window", op="paged", dtype="bf16", requests=128, idle=0, new=1, chunks=0,
             context=4000, longest=32768, ctx_seed=2, H=16, Hkv=4, D=64, page=16, window=1024, sinks=4),
        # a prompt's later chunk beside requests that decode
        dict(name="paged_chunk_mixed", op="paged", dtype="bf16", requests=21, idle=0, new=2048, chunks=1,
             context=2000, longest=30001, ctx_seed=3, H=32, Hkv=8, D=128, page=64, window=0, sinks=0),
        # a prompt's keys and values into the cache
        dict(name="append_chunk", op="append", dtype="bf16", requests=4, idle=0, new=2000, chunks=4, context=3000,
             longest=16384, ctx_seed=4, Hkv=8, D=128, page=16),
        # those of a decoding step: the call's latency
        dict(name="append_decode", op="append", dtype="bf16", requests=64, idle=3, new=1, chunks=0, context=2000,
             longest=16384, ctx_seed=1, Hkv=8, D=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "window", "window", "window", "paged", "paged", "paged", "append"])
    f32 = rng.random() < 0.15
    dtype, D = ("f32", rng.choice([32, 64, 128])) if f32 else ("bf16", rng.choice([64, 128]))
    Hkv = rng.choice([1, 2, 3, 4] if f32 else [1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4])
    seed = rng.randint(1, 1 << 20)
    if op == "norm_rope":
        train = rng.random() < 0.5
        return dict(op=op, train=train, dtype=dtype, tokens=_log_int(rng, 1, 16384 if train else 65536),
                    docs=rng.choice(["lognormal", "uniform", "one"]), median=rng.randint(30, 2000), doc_seed=seed,
                    H=H, Hkv=Hkv, D=D, rot=16 * rng.randint(1, D // 16), interleaved=rng.random() < 0.3,
                    fused=rng.random() < 0.5, far=rng.choice([0, _log_int(rng, 1, 1 << 20)]))
    if op == "window":
        train = rng.random() < 0.5
        docs = rng.choice(["lognormal", "uniform", "one"])
        if f32:
            tokens, docs = _log_int(rng, 48, 1024), rng.choice(["uniform", "one"])
        else:
            tokens = _log_int(rng, 33, 16384 if train else 32768)
        if docs == "one":
            tokens = min(tokens, 12000)
        case = dict(op=op, train=train, dtype=dtype, tokens=tokens,
                    tail=0 if docs == "one" else rng.choice([0, rng.randint(0, tokens // 8)]), docs=docs,
                    median={"lognormal": rng.randint(200, 2000), "uniform": rng.randint(30, 300), "one": 0}[docs],
                    doc_seed=seed, max_segs=0, H=H, Hkv=Hkv, D=D, window=_log_int(rng, 8, 2048),
                    sinks=rng.choice([0, 0, 1, 4, rng.randint(2, 64)]))
        case["max_segs"] = len(_lengths(case)) + rng.randint(0, 9)
        return case
    case = dict(op=op, dtype=dtype, requests=_log_int(rng, 1, 24 if f32 else 96), idle=0, new=1, chunks=0,
                context=_log_int(rng, 16, 2000 if f32 else 6000), longest=0, ctx_seed=seed, H=H, Hkv=Hkv, D=D,
                page=rng.choice([16, 32, 64, 128]), window=0, sinks=0)
    case["longest"] = case["context"] * rng.randint(1, 6)
    case["idle"] = rng.randint(0, case["requests"] // 8)
    if rng.random() < 0.5:
        case["chunks"] = rng.randint(1, max(1, min(case["requests"] - case["idle"], 4)))
        case["new"] = _log_int(rng, 2, 200 if f32 else 1500)
    if rng.random() < 0.4:
        case["window"], case["sinks"] = _log_int(rng, 8, 2048), rng.choice([0, 4, rng.randint(1, 64)])
    if op == "append":
        for name in ("H", "window", "sinks"):
            del case[name]
    return case


def _lengths(case):
    """Document lengths of a case (they fill tokens - tail)."""
    room = case["tokens"] - case.get("tail", 0)
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


def _requests(case):
    """(cached tokens, new tokens) of every request; an idle one has (0, 1): a row of the batch that sees nothing."""
    rng = random.Random(case["ctx_seed"])
    out = []
    for r in range(case["requests"]):
        if r < case["chunks"]:
            n = case["new"] if case["chunks"] == 1 else rng.randint(case["new"] // 2 + 1, case["new"] + 100)
            out.append((max(0, case["longest"] - n) if r == 0 else rng.randint(0, case["context"]), n))
        elif case["requests"] - r <= case["idle"]:
            out.append((0, 1))
        elif case["requests"] == 1:
            out.append((case["longest"] - 1, 1))
        else:
            n = int(round(case["context"] * math.exp(rng.gauss(0.0, 0.8))))
            out.append((min(max(n, 1), case["longest"]), 1))
    return out


def _visible(ctx, n, window, sinks):
    """Query-key pairs of n new tokens behind ctx cached ones, and the keys that any of them sees."""
    if window <= 0:
        return n * ctx + n * (n + 1) // 2, ctx + n
    pairs = sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(ctx, ctx + n))
    low = max(0, ctx - window + 1)
    return pairs, ctx + n - low + min(sinks, low)


# ---------------------------------------------------------------- the inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    dt, D, Hkv = _DTYPES[case["dtype"]], case["D"], case["Hkv"]
    if case["op"] == "norm_rope":
        N, H, rot = case["tokens"], case["H"], case["rot"]
        if case["fused"]:
            qkv = _normal(gen, (1, N, H + 2 * Hkv, D), dt)
            st["q"], st["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        else:
            st["q"], st["k"] = _normal(gen, (1, N, H, D), dt), _normal(gen, (1, N, Hkv, D), dt)
        for x in ("q", "k"):
            st["w" + x] = 1.0 + 0.2 * _normal(gen, (D,), torch.float32)
            if case["train"]:
                st["d" + x] = _normal(gen, (1, N, H if x == "q" else Hkv, D), dt)
        lens = _lengths(case)
        far = 0 if case["far"] == 0 else seed % case["far"]
        pos = np.concatenate([far + np.arange(n) for n in lens])[:N].astype(np.int32)
        st["pos"] = torch.from_numpy(pos).cuda()
        st["freq"] = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)).cuda()
        return st
    if case["op"] == "window":
        N, H = case["tokens"], case["H"]
        st["lens"] = lens = _lengths(case)
        cu = np.full(case["max_segs"] + 1, sum(lens), dtype=np.int32)
        cu[:len(lens) + 1] = np.concatenate([[0], np.cumsum(lens)])
        st["cu"] = torch.from_numpy(cu).cuda()
        st["q"], st["k"], st["v"] = (_normal(gen, (1, N, h, D), dt) for h in (H, Hkv, Hkv))
        if case["train"]:
            st["do"] = _normal(gen, (1, N, H, D), dt)
        return st
    st["reqs"] = reqs = _requests(case)
    page, append = case["page"], case["op"] == "append"
    N = sum(n for _, n in reqs)
    total = [0 if idle else c + n for (c, n), idle in zip(reqs, _idle(case))]
    need = [-(-t // page) for t in total]
    spare = 5
    pages = np.random.default_rng(seed).permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(reqs), max(need) + 2), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = pages[at:at + n]
        at += n
    st["table"], st["lens"] = torch.from_numpy(table).cuda(), torch.tensor(total, dtype=torch.int32).cuda()
    cu = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    st["cu"] = torch.from_numpy(cu).cuda() if case["chunks"] else None
    st["kc"], st["vc"] = (_normal(gen, (len(pages), page, Hkv, D), dt) for _ in range(2))
    if append:
        st["k"], st["v"] = _normal(gen, (N, Hkv, D), dt), _normal(gen, (N, Hkv, D), dt)
    else:
        st["q"] = _normal(gen, (N, case["H"], D), dt)
    return st


def _idle(case):
    return [r >= case["chunks"] and case["requests"] - r <= case["idle"] for r in range(case["requests"])]


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_norm_rope(st):
    import packed_varlen_gated_amd as pkv
    case = st["case"]
    args = (st["wq"], st["wk"], st["pos"], st["freq"], _EPS, case["interleaved"])
    q, k = pkv.qk_norm_rope(st["q"], st["k"], *args)
    out = {"q": q, "k": k}
    if case["train"]:
        gr = pkv.qk_norm_rope_backward(st["q"], st["k"], st["dq"], st["dk"], *args)
        out.update(dq=gr.dq, dk=gr.dk, dwq=gr.dq_weight, dwk=gr.dk_weight)
    return out


def _own_window(st):
    import packed_varlen_gated_amd as pkv
    case = st["case"]
    vis = (case["window"], case["sinks"], st["cu"])
    o, lse = pkv.attn_window_varlen(st["q"], st["k"], st["v"], *vis, output_lse=case["train"])
    if not case["train"]:
        return {"o": o}
    gr = pkv.attn_window_varlen_backward(st["q"], st["k"], st["v"], o, lse, st["do"], *vis)
    return {"o": o, "dq": gr.dq, "dk": gr.dk, "dv": gr.dv}


def _own_paged(st):
    import packed_varlen_gated_amd as pkv
    case = st["case"]
    o, _ = pkv.attn_paged(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["cu"],
                          window=case["window"] or None, sinks=case["sinks"])
    return {"o": o}


def _own_append(st):
    import packed_varlen_gated_amd as pkv
    pkv.paged_kv_append(st["k"], st["v"], st["kc"], st["vc"], st["table"], st["lens"], st["cu"])
    return {"k": st["kc"], "v": st["vc"]}


_OWN = {"norm_rope": _own_norm_rope, "window": _own_window, "paged": _own_paged, "append": _own_append}


# Plain forms.

def _pairs(x, rot, interleaved):
    """The two members of every rotated pair, and the channels that are not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _plain_norm_rope(st):
    case = st["case"]
    rot, il = case["rot"], case["interleaved"]
    # (angles of far positions lose their fraction in 32 bits)
    angle = st["pos"].double()[:, None] * st["freq"].double()[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = {}
    for x in ("q", "k"):
        u = st[x][0].float()
        r = 1.0 / torch.sqrt(u.square().mean(-1, keepdim=True) + _EPS)
        u = u * r
        a, b, rest = _pairs(u * st["w" + x], rot, il)
        out[x] = _unpairs(a * cos - b * sin, a * sin + b * cos, rest, il)[None].to(st[x].dtype)
        if not case["train"]:
            continue
        a, b, rest = _pairs(st["d" + x][0].float(), rot, il)
        d = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, il)
        out["dw" + x] = (d * u).sum((0, 1))
        d = d * st["w" + x]
        out["d" + x] = (r * (d - u * (d * u).mean(-1, keepdim=True)))[None].to(st[x].dtype)
    return out


# Documents, or requests, of similar length are padded to one batch.

def _batches(lens, cost):
    """Groups of indices of lengths within a factor of two; cost(longest): score elements of one member."""
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    i = 0
    while i < len(order):
        L = lens[order[i]]
        n = max(1, min(len(order) - i, _SCORES // max(cost(L), 1)))
        grp = [order[j] for j in range(i, i + n) if lens[order[j]] * 2 >= L]
        i += len(grp)
        yield grp, L


def _mask(tq, tk, window, sinks):
    """Which keys (places tk [.., L]) the queries (places tq [.., n]) see."""
    gap = tq[..., :, None] - tk[..., None, :]
    see = gap >= 0
    if window > 0:
        see = see & ((gap < window) | (tk[..., None, :] < sinks))
    return see


def _softmax(Q, K, see, scale):
    """Q [G, h, rep, n, D], K [G, h, L, D], see [G or 1, n, L] -> weights [G, h, rep n, L]; a row that sees
    nothing has none."""
    G, h, rep, n, D = Q.shape
    S = torch.matmul(Q.reshape(G, h, rep * n, D), K.transpose(-1, -2).contiguous()).view(G, h, rep, n, -1) * scale
    S = S.masked_fill(~see[:, None, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    S = torch.exp(S - top.masked_fill(top == -math.inf, 0.0))
    return (S / S.sum(-1, keepdim=True).clamp_min(1e-37)).view(G, h, rep * n, -1)


def _plain_window(st):
    case = st["case"]
    H, Hkv, D, train = case["H"], case["Hkv"], case["D"], case["train"]
    rep, scale = H // Hkv, 1.0 / math.sqrt(D)
    x = {n: st[n][0] for n in ("q", "k", "v") + (("do",) if train else ())}
    out = {"o": torch.zeros_like(x["q"])}
    if train:
        out.update(dq=torch.zeros_like(x["q"]), dk=torch.zeros_like(x["k"]), dv=torch.zeros_like(x["v"]))
    starts = np.concatenate([[0], np.cumsum(st["lens"])])
    for grp, L in _batches(st["lens"], lambda L: H * L * L):
        t = torch.arange(L)
        n = torch.tensor([st["lens"][i] for i in grp])[:, None]
        idx = (torch.tensor([int(starts[i]) for i in grp])[:, None] + torch.minimum(t[None], n - 1)).cuda()
        real = (t[None] < n).cuda()
        G, t = len(grp), t.cuda()
        see = _mask(t, t, case["window"], case["sinks"])[None]
        get = lambda a, h: (a[idx].float() * real[:, :, None, None]).transpose(1, 2).reshape(G, Hkv, h, L, D)

        def put(a, y):
            a[idx[real]] = y.reshape(G, -1, L, D).transpose(1, 2)[real].to(a.dtype)
        Q, K, V = get(x["q"], rep), get(x["k"], 1)[:, :, 0], get(x["v"], 1)[:, :, 0]
        O = torch.empty_like(Q)
        if train:
            DO, DQ, DK, DV = get(x["do"], rep), torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
        step = max(1, min(Hkv, _SCORES // max(1, G * rep * L * L)))
        for a in range(0, Hkv, step):
            b = min(Hkv, a + step)
            rows = lambda y: y[:, a:b].reshape(G, b - a, rep * L, D)
            P = _softmax(Q[:, a:b], K[:, a:b], see, scale)
            Oh = torch.matmul(P, V[:, a:b])
            O[:, a:b] = Oh.view(G, b - a, rep, L, D)
            if train:
                d = rows(DO)
                DV[:, a:b] = torch.matmul(P.transpose(-1, -2), d)
                DS = P * (torch.matmul(d, V[:, a:b].transpose(-1, -2).contiguous()) - (d * Oh).sum(-1, keepdim=True))
                DQ[:, a:b] = (torch.matmul(DS, K[:, a:b]) * scale).view(G, b - a, rep, L, D)
                DK[:, a:b] = torch.matmul(DS.transpose(-1, -2), rows(Q)) * scale
        put(out["o"], O)
        if train:
            put(out["dq"], DQ)
            put(out["dk"], DK)
            put(out["dv"], DV)
    return {n: y[None] for n, y in out.items()}


def _plain_paged(st):
    case = st["case"]
    H, Hkv, D, page = case["H"], case["Hkv"], case["D"], case["page"]
    rep, scale = H // Hkv, 1.0 / math.sqrt(D)
    o = torch.zeros_like(st["q"])
    starts = np.concatenate([[0], np.cumsum([n for _, n in st["reqs"]])])
    ones = [r for r in range(len(st["reqs"])) if st["reqs"][r][1] == 1]
    groups = [([ones[i] for i in grp], 1) for grp, _ in
              _batches([sum(st["reqs"][r]) for r in ones], lambda L: 2 * Hkv * D * L)]
    groups += [([r], n) for r, (_, n) in enumerate(st["reqs"]) if n > 1]
    for grp, n in groups:
        G = len(grp)
        L = max(sum(st["reqs"][r]) for r in grp)
        rows = torch.tensor(grp).cuda()
        pages = st["table"][rows, :-(-L // page)].clamp_min(0).long()
        K, V = (c[pages].flatten(1, 2)[:, :L].float().transpose(1, 2) for c in (st["kc"], st["vc"]))
        lens = st["lens"][rows].long()[:, None]
        tk = torch.arange(L, device="cuda")[None]
        at = torch.tensor([int(starts[r]) for r in grp])[:, None].cuda() + torch.arange(n, device="cuda")[None]
        V = V.masked_fill((tk >= lens)[:, None, :, None], 0.0)     # what the pages hold behind the last token
        see = _mask(lens - n + torch.arange(n, device="cuda")[None], tk.expand(G, -1), case["window"], case["sinks"])
        Q = st["q"][at].float().transpose(1, 2).reshape(G, Hkv, rep, n, D)
        O = torch.empty_like(Q)
        step = max(1, min(Hkv, _SCORES // (G * rep * n * L)))
        for a in range(0, Hkv, step):
            P = _softmax(Q[:, a:a + step], K[:, a:a + step], see, scale)
            O[:, a:a + step] = torch.matmul(P, V[:, a:a + step]).view(G, -1, rep, n, D)
        o[at] = O.view(G, H, n, D).transpose(1, 2).to(o.dtype)
    return {"o": o}


def _plain_append(st):
    case = st["case"]
    n = torch.tensor([n for _, n in st["reqs"]]).cuda()
    r = torch.repeat_interleave(torch.arange(len(st["reqs"]), device="cuda"), n)
    first = torch.cumsum(n, 0) - n
    place = st["lens"].long()[r] - n[r] + torch.arange(len(r), device="cuda") - first[r]
    ok = place >= 0
    r, place = r[ok], place[ok]
    page = st["table"][r, place // case["page"]].long()
    for x, c in (("k", "kc"), ("v", "vc")):
        st[c][page, place % case["page"]] = st[x][ok]
    return {"k": st["kc"], "v": st["vc"]}


_PLAIN = {"norm_rope": _plain_norm_rope, "window": _plain_window, "paged": _plain_paged, "append": _plain_append}


# ---------------------------------------------------------------- the work

def work(case):
    """Every input read once, every output written once (of the cache the keys and values that are seen, or the
    places that are written); the products of the visible pairs."""
    es = 2 if case["dtype"] == "bf16" else 4
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "norm_rope":
        x = case["tokens"] * (case["H"] + Hkv) * D
        if not case["train"]:
            return {"bytes": 2 * x * es + case["tokens"] * 4, "flops": 8 * x}
        return {"bytes": 5 * x * es + case["tokens"] * 8, "flops": 24 * x}
    if case["op"] == "window":
        lens = _lengths(case)
        pairs = sum(_visible(0, n, case["window"], case["sinks"])[0] for n in lens)
        q, kv = sum(lens) * case["H"] * D * es, sum(lens) * Hkv * D * es
        if not case["train"]:
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * D * case["H"] * pairs}
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * D * case["H"] * pairs}
    live = [x for x, idle in zip(_requests(case), _idle(case)) if not idle]
    new = sum(n for _, n in live)
    if case["op"] == "append":
        return {"bytes": 4 * new * Hkv * D * es, "flops": 0}
    seen = [_visible(c, n, case["window"], case["sinks"]) for c, n in live]
    return {"bytes": 2 * sum(k for _, k in seen) * Hkv * D * es + 2 * new * case["H"] * D * es,
            "flops": 4 * D * case["H"] * sum(p for p, _ in seen)}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "window": _exact_window, "paged": _exact_paged,
            "append": _exact_append}[case["op"]](st)


def _exact_norm_rope(st):
    """Every pair as a complex number times e^{i angle}; the gradients by differentiating it, some tokens at a
    time."""
    case = st["case"]
    rot, out = case["rot"], {}
    for x in ("q", "k"):
        N, h, D = st[x].shape[1:]
        y = torch.empty(N, h, D, dtype=torch.float64, device="cuda")
        w = st["w" + x].double().requires_grad_(case["train"])
        dx, dw = torch.empty_like(y) if case["train"] else None, torch.zeros_like(w)
        for a in range(0, N, 4096):
            e = min(N, a + 4096)
            u = st[x][0, a:e].double().requires_grad_(case["train"])
            z = w * u * torch.rsqrt((u * u).mean(-1, keepdim=True) + _EPS)
            turned = z[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
            first, second = turned.unbind(-1 if case["interleaved"] else -2)
            phase = torch.outer(st["pos"][a:e].double(), st["freq"].double())[:, None]
            c = torch.complex(first, second) * torch.polar(torch.ones_like(phase), phase)
            both = torch.stack([c.real, c.imag], -1 if case["interleaved"] else -2).flatten(-2)
            part = torch.cat([both, z[..., rot:]], -1)
            y[a:e] = part.detach()
            if case["train"]:
                g = torch.autograd.grad(part, [u, w], st["d" + x][0, a:e].double())
                dx[a:e] = g[0]
                dw = dw + g[1]
        out[x] = y[None]
        if case["train"]:
            out["d" + x], out["dw" + x] = dx[None], dw
    return out


def _exact_window(st):
    """Rows of a document in blocks, with the keys that any of them sees; the gradients by differentiating it."""
    case = st["case"]
    rep, D, train, W, S = case["H"] // case["Hkv"], case["D"], case["train"], case["window"], case["sinks"]
    full = {n: torch.zeros(st[s].shape, dtype=torch.float64, device="cuda")
            for n, s in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")) if train or n == "o"}
    a = 0
    for n in st["lens"]:
        for r in range(0, n, 1024):
            e = min(n, r + 1024)
            low = max(0, r - W + 1)
            keys = torch.cat([torch.arange(min(S, low)), torch.arange(low, e)]).cuda()
            t = torch.arange(r, e, device="cuda")[:, None]
            hidden = (keys > t) | ((keys <= t - W) & (keys >= S))
            for h in range(case["Hkv"]):
                hs = slice(h * rep, (h + 1) * rep)
                q = st["q"][0, a + r:a + e, hs].double().requires_grad_(train)
                k, v = (st[x][0, a + keys, h].double().requires_grad_(train) for x in ("k", "v"))
                s = torch.matmul(q.transpose(0, 1), k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                o = torch.matmul(torch.softmax(s, -1), v).transpose(0, 1)
                full["o"][0, a + r:a + e, hs] = o.detach()
                if train:
                    d = torch.autograd.grad(o, [q, k, v], st["do"][0, a + r:a + e, hs].double())
                    full["dq"][0, a + r:a + e, hs] = d[0]
                    full["dk"][0, a + keys, h] += d[1]
                    full["dv"][0, a + keys, h] += d[2]
        a += n
    return full


def _exact_paged(st):
    """Request by request and query by query (or a block of them): the softmax over its visible places."""
    case = st["case"]
    rep, D, page, W, S = case["H"] // case["Hkv"], case["D"], case["page"], case["window"], case["sinks"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r, (_, n) in enumerate(st["reqs"]):
        total = int(st["lens"][r])
        if total:
            places = torch.arange(total, device="cuda")
            where = st["table"][r, places // page].long() * page + places % page
            for a in range(0, n, 256):
                e = min(n, a + 256)
                t = total - n + torch.arange(a, e, device="cuda")[:, None]
                hidden = places > t
                if W > 0:
                    hidden = hidden | ((places <= t - W) & (places >= S))
                for h in range(case["Hkv"]):
                    k, v = (st[c].flatten(0, 1)[where, h].double() for c in ("kc", "vc"))
                    q = st["q"][at + a:at + e, h * rep:(h + 1) * rep].double().transpose(0, 1)
                    p = torch.softmax(torch.matmul(q, k.T / math.sqrt(D)).masked_fill(hidden, -math.inf), -1)
                    out[at + a:at + e, h * rep:(h + 1) * rep] = torch.matmul(p, v).transpose(0, 1)
        at += n
    return {"o": out}


def _exact_append(st):
    """Token by token (values are copied: the result is their own type's)."""
    case = st["case"]
    table, lens = st["table"].cpu(), st["lens"].cpu()
    at = 0
    for r, (_, n) in enumerate(st["reqs"]):
        for j in range(n):
            p = int(lens[r]) - n + j
            if p >= 0:
                pg, i = int(table[r, p // case["page"]]), p % case["page"]
                st["kc"][pg, i] = st["k"][at + j]
                st["vc"][pg, i] = st["v"][at + j]
        at += n
    return {"k": st["kc"].double(), "v": st["vc"].double()}
