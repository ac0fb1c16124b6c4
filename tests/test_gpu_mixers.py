"""The packed mixers and the single-token steps on the GPU against the fp64
oracle, with the bounds of mixer_parity.py, and their invariants bit by bit."""

import numpy as np
import pytest
import torch

import packed_varlen_gated_amd as pkv
from mixer_parity import attn_bounds, check, gamma, half_step, linear_bounds
from oracle import mixers

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LENS = {
    "one": [1],
    "singles": [1, 1, 1],
    "edges": [31, 32, 33, 63, 64, 65, 1],
    "tiles": [127, 128, 129, 0, 0, 17],
    "long": [0, 385, 5, 700],
}
TAIL = {"one": 0, "singles": 2, "edges": 0, "tiles": 13, "long": 70}


def dev():
    return torch.device("cuda", 0)


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def lay(lens, tail):
    cu = np.concatenate([[0], np.cumsum(lens)])
    return int(cu[-1]) + tail, cu


def on_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype]).to(dev())


def cu_gpu(cu):
    return torch.from_numpy(np.asarray(cu).astype(np.int32)).to(dev())


def attn_inputs(seed, N, Hq, Hkv, D, dtype, amp=1.0):
    rng = np.random.default_rng(seed)
    return [on_gpu(rng.standard_normal((1, N, h, D)) * a, dtype) for h, a in ((Hq, amp), (Hkv, amp), (Hkv, 1), (Hq, 1))]


def linear_inputs(seed, N, H, Dk, Dv, dtype, segs=0):
    rng = np.random.default_rng(seed)
    q, k = (rng.standard_normal((1, N, H, Dk)) / np.sqrt(Dk) for _ in range(2))
    v, do = (rng.standard_normal((1, N, H, Dv)) for _ in range(2))
    g = torch.tensor([-0.7 * 0.5 ** h if h else 0.0 for h in range(H)], dtype=torch.float32, device=dev())
    st = [torch.from_numpy(rng.standard_normal((segs, H, Dk, Dv))).float().to(dev()) for _ in range(2)] if segs else [None, None]
    return [on_gpu(x, dtype) for x in (q, k, v, do)] + [g] + st


def attn_run(q, k, v, do, cud, scale=None):
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, lse = pkv.attn_varlen(q, k, v, cud, scale, flags=flags)
    gr = pkv.attn_varlen_backward(q, k, v, o, lse, do, cud, scale, flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    return dict(o=o, lse=lse, dq=gr.dq, dk=gr.dk, dv=gr.dv)


def attn_case(lens, tail, Hq, Hkv, D, dtype, seed=0, scale=None, amp=1.0, none=False):
    N, cu = lay(lens, tail)
    q, k, v, do = attn_inputs(seed, N, Hq, Hkv, D, dtype, amp)
    got = attn_run(q, k, v, do, None if none else cu_gpu(cu), scale)
    want = attn_bounds(host(q)[0], host(k)[0], host(v)[0], host(do)[0], None if none else cu, scale, dtype)
    end = int(cu[-1])
    for name, (ref, bound, extra) in want.items():
        x = host(got[name])
        if name == "lse":
            assert (x[:, end:] == -np.inf).all()
            check(x[:, :end], ref[:, :end], bound[:, :end], "f32", name)
        else:
            assert not x[0, end:].any(), name
            check(x[0], ref, bound, dtype, name, extra)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("case", list(LENS))
def test_attn(case, dtype, D):
    attn_case(LENS[case], TAIL[case], 4, 2, D, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 1), (8, 2), (5, 5)])
@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_attn_heads(Hq, Hkv, dtype, D):
    attn_case([70, 130], 3, Hq, Hkv, D, dtype, seed=Hq)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_attn_one_segment_and_scales(dtype, D):
    attn_case([200], 0, 2, 1, D, dtype, none=True)
    attn_case([200], 0, 2, 1, D, dtype, scale=-0.3)          # a negative scale
    attn_case([200], 0, 2, 1, D, dtype, scale=0.0)           # equal weights
    attn_case([300, 90], 0, 2, 1, D, dtype, amp=4.0)         # sharp weights


@pytest.mark.parametrize("D", [64, 128])
def test_attn_many_tiles(D):
    attn_case([1500, 300, 2], 7, 2, 1, D, "bf16", seed=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 1), (4, 2), (20, 10)])
def test_attn_one_long_segment_among_short_ones(Hq, Hkv, D):
    """The keys pass whose waves share keys is chosen by the longest segment; the short ones go through it too."""
    attn_case([33, 0, 1100, 1, 63, 64, 65, 0, 129, 31], 40, Hq, Hkv, D, "bf16", seed=Hq + D)
    attn_case([3] * 70 + [1000] + [0] * 200, 0, Hq, Hkv, D, "bf16", seed=D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,tail", [(1024, 0), (1087, 0), (1050, 130)])
def test_attn_one_segment_of_many_tiles(N, tail, D):
    """A single segment with few heads: waves share queries in the forward pass, 64 keys each."""
    attn_case([N - 63 * (tail > 0)], tail, 4, 2, D, "bf16", seed=N + D)
    attn_case([N], 0, 2, 2, D, "bf16", seed=N, scale=-0.2, amp=3.0, none=True)
    # a later token's values reach no earlier row
    q, k, v, do = attn_inputs(N, N, 2, 1, D, "bf16")
    o, lse = pkv.attn_varlen(q, k, v)
    for a in (N - 1, 700, 64):
        x = [t.clone() for t in (q, k, v)]
        for t in x:
            t[0, a:a + 9] = float("nan")
        y, z = pkv.attn_varlen(*x)
        assert torch.equal(y[0, :a], o[0, :a]) and torch.equal(z[:, :a], lse[:, :a]), a


@pytest.mark.parametrize("D", [64, 128])
def test_attn_none_is_one_segment(D):
    """Without cu_seqlens the form of the keys pass is chosen on the host, with it on the device: the same one."""
    for N in (100, 700, 1300):
        q, k, v, do = attn_inputs(N, N, 2, 1, D, "bf16")
        a, b = attn_run(q, k, v, do, None), attn_run(q, k, v, do, cu_gpu([0, N]))
        assert all(torch.equal(a[n], b[n]) for n in a), N


def test_attn_captured_with_changing_lengths():
    """A captured reverse pass goes by the lengths that cu_seqlens holds at the replay."""
    N, D = 1300, 64
    q, k, v, do = attn_inputs(23, N, 4, 2, D, "bf16")
    lays = [[0, 1300, 1300, 1300, 1300], [0, 200, 500, 800, 1100], [0, 1, 1290, 1290, 1295], [0, 0, 0, 0, 0]]
    want = [attn_run(q, k, v, do, cu_gpu(c)) for c in lays]
    cud = cu_gpu(lays[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o, lse = pkv.attn_varlen(q, k, v, cud)
        pkv.attn_varlen_backward(q, k, v, o, lse, do, cud)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = pkv.attn_varlen(q, k, v, cud)
        gr = pkv.attn_varlen_backward(q, k, v, o, lse, do, cud)
    for i in (0, 1, 2, 3, 1, 0):
        cud.copy_(cu_gpu(lays[i]))
        g.replay()
        torch.cuda.synchronize()
        for n, x in dict(o=o, lse=lse, dq=gr.dq, dk=gr.dk, dv=gr.dv).items():
            assert torch.equal(x, want[i][n]), (i, n)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_attn_segments_are_isolated(dtype, D):
    """NaN and infinities in one segment and behind the last reach no other: the bits stay."""
    N, cu = lay([90, 60, 140], 40)
    q, k, v, do = attn_inputs(3, N, 4, 2, D, dtype)
    ref = attn_run(q, k, v, do, cu_gpu(cu))
    for t in (q, k, v, do):
        t[0, 90:150] = float("nan")
        t[0, 120] = float("inf")
        t[0, 290:] = float("nan")
    got = attn_run(q, k, v, do, cu_gpu(cu))
    for name in ref:
        for sl in (slice(0, 90), slice(150, 290)):
            x, y = (r[name][:, sl] if name == "lse" else r[name][0, sl] for r in (got, ref))
            assert torch.equal(x, y), name
    assert not got["o"][0, 290:].any() and not got["dv"][0, 290:].any()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_attn_later_tokens_do_not_reach_earlier_ones(dtype, D):
    """Padding that joined a segment's tail may hold anything: the tokens before it keep their bits."""
    N, cu = lay([100, 333], 0)
    q, k, v, do = attn_inputs(4, N, 4, 2, D, dtype)
    ref, rl = pkv.attn_varlen(q, k, v, cu_gpu(cu))
    for bad in (float("nan"), float("inf"), -float("inf")):
        for a, e in ((77, 100), (417, 433), (140, 433)):
            k2, v2 = k.clone(), v.clone()
            k2[0, a:e] = bad
            v2[0, a:e] = bad
            o, lse = pkv.attn_varlen(q, k2, v2, cu_gpu(cu))
            keep = torch.ones(N, dtype=torch.bool, device=dev())
            keep[a:(100 if a < 100 else 433)] = False
            assert torch.equal(o[0][keep], ref[0][keep]) and torch.equal(lse[:, keep], rl[:, keep]), (bad, a)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_attn_equal_calls_give_equal_bits(dtype, D):
    N, cu = lay([200, 57, 300], 9)
    q, k, v, do = attn_inputs(6, N, 4, 2, D, dtype)
    a, b = (attn_run(q, k, v, do, cu_gpu(cu)) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    # without lse the output is the same
    assert torch.equal(pkv.attn_varlen(q, k, v, cu_gpu(cu), output_lse=False)[0], a["o"])


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_attn_packed_equals_alone(dtype, D):
    N, cu = lay([200, 57, 300], 0)
    q, k, v, do = attn_inputs(7, N, 4, 2, D, dtype)
    all_ = attn_run(q, k, v, do, cu_gpu(cu))
    for a, e in zip(cu[:-1], cu[1:]):
        one = attn_run(*(t[:, a:e].contiguous() for t in (q, k, v, do)), None)
        for n in one:
            x = all_[n][:, a:e] if n == "lse" else all_[n][0, a:e]
            assert torch.equal(x, one[n] if n == "lse" else one[n][0]), n


@pytest.mark.parametrize("bad", [[1, 5, 20], [0, 30, 20], [0, 10, 50], [-3, 10, 20], [0, 100, 20]])
def test_bad_cu_seqlens_set_the_flag(bad):
    q, k, v, do = attn_inputs(8, 40, 2, 2, 64, "bf16")
    cu = cu_gpu(bad)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, lse = pkv.attn_varlen(q, k, v, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS
    flags.zero_()
    pkv.attn_varlen_backward(q, k, v, o, lse, do, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS
    g = torch.zeros(2, device=dev())
    flags.zero_()
    pkv.chunk_linear_attn_varlen(q, k, v, g, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS
    flags.zero_()
    pkv.chunk_linear_attn_varlen_backward(q, k, v, g, do, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS


def test_many_empty_slots():
    """Slots far beyond 64 x 64, most of them empty."""
    lens = [0] * 4500 + [70] + [0] * 300 + [33, 1] + [0] * 77
    attn_case(lens, 5, 2, 1, 64, "bf16")
    linear_case(lens, 5, 2, 64, 64, "bf16", states=False)


@pytest.mark.parametrize("D", [64, 128])
def test_attn_short_segments_many_heads(D):
    """Enough slots and heads that a work-group takes several heads of its tile (10 heads: groups of 4, 4, 2)."""
    rng = np.random.default_rng(17)
    lens = []
    while sum(lens) < 13300:
        lens.append(int(rng.integers(1, 260)))
    lens[3:3] = [0] * 600
    attn_case(lens, 21, 10, 10, D, "bf16", seed=18)
    N, cu = lay(lens, 21)
    q, k, v, do = attn_inputs(19, N, 10, 10, D, "bf16")
    ref = attn_run(q, k, v, do, cu_gpu(cu))
    for t in (q, k, v, do):
        t[0, cu[605] + 1:cu[606]] = float("nan")     # a segment's later tokens
    got = attn_run(q, k, v, do, cu_gpu(cu))
    keep = torch.ones(N, dtype=torch.bool, device=dev())
    keep[cu[605] + 1:cu[606]] = False
    assert torch.equal(got["o"][0][keep], ref["o"][0][keep])
    keep[cu[605]:cu[606]] = False
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n][0][keep], ref[n][0][keep]), n


# ------------------------------------------------------- linear attention

def linear_run(q, k, v, do, g, S0, dF, cud, scale=1.0):
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, fs = pkv.chunk_linear_attn_varlen(q, k, v, g, cud, scale, initial_state=S0, flags=flags)
    gr = pkv.chunk_linear_attn_varlen_backward(q, k, v, g, do, cud, scale, initial_state=S0, dfinal_state=dF,
                                               output_d_initial_state=True, flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    return dict(o=o, final=fs, dq=gr.dq, dk=gr.dk, dv=gr.dv, dinit=gr.d_initial_state)


def linear_case(lens, tail, H, Dk, Dv, dtype, states, seed=0, scale=1.0, none=False, g=None):
    N, cu = lay(lens, tail)
    q, k, v, do, g0, S0, dF = linear_inputs(seed, N, H, Dk, Dv, dtype, len(lens) if states else 0)
    g = g0 if g is None else torch.tensor(g, dtype=torch.float32, device=dev())
    got = linear_run(q, k, v, do, g, S0, dF, None if none else cu_gpu(cu), scale)
    want = linear_bounds(host(q)[0], host(k)[0], host(v)[0], host(g), host(do)[0], None if none else cu, scale,
                         host(S0), host(dF), dtype)
    end = int(cu[-1])
    for name, (ref, bound) in want.items():
        x = host(got[name])
        if name in ("final", "dinit"):
            check(x, ref, bound, "f32", name)
        else:
            assert not x[0, end:].any(), name
            check(x[0], ref, bound, dtype, name)


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("dtype,Dk,Dv", [("f32", 32, 32), ("f32", 64, 128), ("bf16", 32, 64), ("bf16", 64, 64),
                                         ("bf16", 64, 128), ("bf16", 128, 64), ("bf16", 128, 128)])
@pytest.mark.parametrize("case", list(LENS))
def test_linear(case, dtype, Dk, Dv, states):
    linear_case(LENS[case], TAIL[case], 3, Dk, Dv, dtype, states, scale=0.5)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_linear_one_segment_and_decays(dtype, D):
    linear_case([200], 0, 3, D, D, dtype, True, none=True)
    linear_case([200], 0, 3, D, D, dtype, True, scale=-2.0)
    linear_case([200, 60], 0, 4, D, D, dtype, True, g=[-1e-4, -3.0, -40.0, 0.0])      # slow, fast, at once, none
    linear_case([150], 0, 1, D, D, dtype, False, g=[-200.0])                          # e^g is 0 in fp32


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_linear_decay_of_minus_infinity_keeps_nothing(dtype, D):
    N, cu = lay([700, 33], 0)
    q, k, v, do, _, _, _ = linear_inputs(23, N, 2, D, D, dtype)
    g = torch.full((2,), -float("inf"), device=dev())
    got = linear_run(q, k, v, do, g, None, None, cu_gpu(cu))
    one = linear_run(q, k, v, do, g, None, None, cu_gpu(np.arange(N + 1)))    # every token alone
    for n in ("o", "dq", "dk", "dv"):
        x, y = host(got[n]), host(one[n])
        # the same products, in another place of a chunk: fp32 sums of D terms, rounded once
        assert np.isfinite(x).all() and np.abs(x - y).max() <= 2 * half_step(dtype) * np.abs(y).max() + gamma(D) * 30


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_linear_many_chunks(D, states):
    linear_case([4500, 3, 1200], 11, 2, D, D, "bf16", states, seed=5)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_linear_segments_are_isolated(dtype, D):
    N, cu = lay([90, 60, 640], 40)
    q, k, v, do, g, S0, dF = linear_inputs(3, N, 3, D, D, dtype, 3)
    ref = linear_run(q, k, v, do, g, S0, dF, cu_gpu(cu))
    for t in (q, k, v, do):
        t[0, 90:150] = float("nan")
        t[0, 120] = float("inf")
        t[0, 790:] = float("nan")
    got = linear_run(q, k, v, do, g, S0, dF, cu_gpu(cu))
    for name in ref:
        for i, sl in ((0, slice(0, 90)), (2, slice(150, 790))):
            x, y = (r[name][i] if name in ("final", "dinit") else r[name][0, sl] for r in (got, ref))
            assert torch.equal(x, y), name
    assert not got["o"][0, 790:].any() and not got["dk"][0, 790:].any()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_linear_equal_calls_give_equal_bits(dtype, D):
    N, cu = lay([200, 57, 1300], 9)
    q, k, v, do, g, S0, dF = linear_inputs(6, N, 3, D, D, dtype, 3)
    a, b = (linear_run(q, k, v, do, g, S0, dF, cu_gpu(cu)) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


# ---------------------------------------------------------------- steps

def step_case(kind, dtype, Dk, Dv, R, S, H, slots, scale=1.0, l2=False, seed=0):
    rng = np.random.default_rng(seed)
    q, k = (on_gpu(rng.standard_normal((R, H, Dk)), dtype) for _ in range(2))
    v = on_gpu(rng.standard_normal((R, H, Dv)), dtype)
    state = torch.from_numpy(rng.standard_normal((S, H, Dk, Dv))).float().to(dev())
    before = state.clone()
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=dev())
    hq, hk = host(q), host(k)
    if kind == "linear":
        g = torch.from_numpy(-rng.uniform(0, 2, H)).float().to(dev())
        o = pkv.linear_attn_step(q, k, v, g, state, sl, scale, flags=flags)
        decay, w = np.exp(host(g))[None, :, None], 1.0
    else:
        g = on_gpu(-rng.uniform(0, 2, (R, H, Dk)), dtype)
        beta = on_gpu(rng.uniform(0, 1, (R, H)), dtype)
        o = pkv.kda_step(q, k, v, g, beta, state, sl, scale, flags=flags, use_qk_l2norm_in_kernel=l2)
        decay, w = np.exp(host(g)), host(beta)
        if l2:
            hq, hk = (x / np.sqrt((x ** 2).sum(-1, keepdims=True) + 1e-6) for x in (hq, hk))
    torch.cuda.synchronize()
    s = list(range(R)) if slots is None else slots
    ro, rs = mixers.step(hq, hk, host(v), decay, w, host(before), s, scale)
    ao, as_ = mixers.step(abs(hq), abs(hk), abs(host(v)), decay, w, abs(host(before)), s, abs(scale))
    f = gamma(Dk + 64)
    check(host(state), rs, f * as_ + 1e-37, "f32", "state")
    check(host(o), ro, f * ao + half_step(dtype) * abs(ro) + 1e-37, "f32", "o")
    untouched = [i for i in range(S) if i not in set(s)]
    assert torch.equal(state[untouched], before[untouched])
    return int(flags)


@pytest.mark.parametrize("kind", ["linear", "kda", "kda_l2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(32, 32), (64, 64), (128, 128), (32, 128), (128, 32), (64, 128)])
def test_step(kind, dtype, Dk, Dv):
    a = dict(kind=kind[:6] if kind == "linear" else "kda", dtype=dtype, Dk=Dk, Dv=Dv, l2=kind == "kda_l2")
    assert step_case(R=1, S=1, H=1, slots=None, **a) == 0
    assert step_case(R=5, S=9, H=3, slots=[8, 0, -1, 3, -7], scale=0.25, **a) == 0


@pytest.mark.parametrize("kind", ["linear", "kda"])
def test_step_bad_and_repeated_slots(kind):
    a = dict(kind=kind, dtype="bf16", Dk=64, Dv=64, H=2)
    assert step_case(R=4, S=3, slots=[0, 3, 1, 1 << 30], **a) == pkv.FLAG_BAD_SLOT
    assert step_case(R=6, S=4, slots=[2, 0, 2, 2, 0, 3], **a) == pkv.FLAG_BAD_SLOT
    assert step_case(R=600, S=700, slots=[-1] * 300 + list(range(300)), **a) == 0
    assert step_case(R=600, S=700, slots=list(range(599)) + [17], **a) == pkv.FLAG_BAD_SLOT


# ------------------------------------------------- used together, and how

@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 32)])
def test_a_packed_model_and_its_decoding(dtype, D):
    """Token rows -> ids -> cu_seqlens -> a softmax layer, then a linear and a KDA layer on its output; the
    recurrent layers' final states continue token by token as a longer prompt would."""
    rng = np.random.default_rng(11)
    H, T, extra = 2, 150, 3
    tokens = rng.integers(1, 9, (1, T)).astype(np.int32)
    tokens[0, [40, 97, T - 1]] = 0
    seg = pkv.eod_to_segment_ids(torch.from_numpy(tokens).to(dev()), 0)
    r = pkv.segment_ids_to_cu_seqlens(seg.segment_ids, 4)
    cu = r.cu_seqlens.cpu().numpy()
    assert cu.tolist() == [0, 41, 98, 150, 150]
    q, k, v, _ = attn_inputs(12, T, H, H, D, dtype)
    x, _ = pkv.attn_varlen(q, k, v, r.cu_seqlens)
    ref, _ = mixers.attn_varlen(host(q)[0], host(k)[0], host(v)[0], cu)
    assert np.linalg.norm(host(x)[0] - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    lq, lk, _, _, g, _, _ = linear_inputs(13, T + extra, H, D, D, dtype)
    g[0] = -0.05
    gates = on_gpu(-rng.uniform(0.01, 0.3, (1, T + extra, H, D)), dtype)
    beta = on_gpu(rng.uniform(0, 1, (1, T + extra, H)), dtype)
    more = on_gpu(rng.standard_normal((1, extra, H, D)), dtype)
    xs = torch.cat([x, more], 1)
    _, fs = pkv.chunk_linear_attn_varlen(lq[:, :T].contiguous(), lk[:, :T].contiguous(), x, g, r.cu_seqlens)
    _, ks = pkv.chunk_kda_varlen(*(t[:, :T].contiguous() for t in (lq, lk, x, gates, beta)), r.cu_seqlens)
    last = torch.tensor([2], dtype=torch.int32, device=dev())
    outs, kouts = [], []
    for t in range(T, T + extra):
        outs.append(pkv.linear_attn_step(lq[0, t:t + 1], lk[0, t:t + 1], xs[0, t:t + 1], g, fs, last))
        kouts.append(pkv.kda_step(lq[0, t:t + 1], lk[0, t:t + 1], xs[0, t:t + 1], gates[0, t:t + 1],
                                  beta[0, t:t + 1], ks, last))
    sl = slice(98, T + extra)
    import oracle
    ro, rfs = mixers.linear_attn_varlen(host(lq)[0, sl], host(lk)[0, sl], host(xs)[0, sl], host(g))
    rk, rks = oracle.chunk_kda_varlen(*(host(t)[0, sl] for t in (lq, lk, xs, gates, beta)), None, 1.0)
    tol = 2.0 ** -8 if dtype == "bf16" else 1e-5
    for got, want, t in ((torch.cat(outs), ro[-extra:], tol), (fs[2], rfs[0], tol),
                         (torch.cat(kouts), rk[-extra:], 2e-2 if dtype == "bf16" else 1e-4),
                         (ks[2], rks[0], 2e-2 if dtype == "bf16" else 1e-4)):
        assert np.linalg.norm(host(got) - want) <= t * np.linalg.norm(want)


def _train_calls(x):
    o, lse = pkv.attn_varlen(x["q"], x["k"], x["v"], x["cu"])
    ga = pkv.attn_varlen_backward(x["q"], x["k"], x["v"], o, lse, x["do"], x["cu"])
    lo, fs = pkv.chunk_linear_attn_varlen(x["q"], x["lk"], x["do"], x["g"], x["cu"])
    gl = pkv.chunk_linear_attn_varlen_backward(x["q"], x["lk"], x["do"], x["g"], o, x["cu"])
    y = pkv.linear_attn_step(x["q"][0, :2], x["lk"][0, :2], x["do"][0, :2], x["g"], fs)
    return [o, lse, *ga, lo, fs, *gl[:3], y]


def _train_inputs(dtype, D, seed):
    N, cu = lay([300, 40, 700], 8)
    q, k, v, do = attn_inputs(seed, N, 4, 2, D, dtype)
    _, lk, _, _, g, _, _ = linear_inputs(seed + 1, N, 4, D, D, dtype)
    return dict(q=q, k=k, v=v, do=do, lk=lk, g=g, cu=cu_gpu(cu))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_captured_and_replayed(dtype, D):
    """Two captured graphs, replayed in turn with new inputs and eager work between, give the eager bits."""
    x = _train_inputs(dtype, D, 21)
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_calls(x)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _train_calls(x)
        graphs.append((g, outs))
    for i in range(5):
        new = _train_inputs(dtype, D, 30 + i)
        for n in x:
            x[n].copy_(new[n])
        want = [t.clone() for t in _train_calls(x)]
        g, outs = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_on_another_stream():
    x = _train_inputs("bf16", 64, 40)
    want = _train_calls(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _train_calls(x)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_past_32_bits(D):
    """Tensors of more than 2^31 elements: the last segment's results equal the segment alone."""
    H, n, last = (256 if D == 64 else 128), 131400, 150
    base = torch.arange(n - last, dtype=torch.int64) // 137 * 137
    cu = torch.unique(base).tolist() + [n - last, n]
    x = {}
    for i, name in enumerate(("q", "k", "v", "do")):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x[name] = torch.empty(1, n, H, D, dtype=torch.bfloat16, device=dev()).normal_(generator=gen)
    assert x["q"].numel() > 1 << 31
    g = torch.full((H,), -0.1, device=dev())
    alone = {m: t[:, n - last:].contiguous() for m, t in x.items()}
    o, lse = pkv.attn_varlen(x["q"], x["k"], x["v"], cu_gpu(cu))
    o1, lse1 = pkv.attn_varlen(alone["q"], alone["k"], alone["v"])
    assert torch.equal(o[:, n - last:], o1) and torch.equal(lse[:, n - last:], lse1)
    gr = pkv.attn_varlen_backward(x["q"], x["k"], x["v"], o, lse, x["do"], cu_gpu(cu))
    gr1 = pkv.attn_varlen_backward(alone["q"], alone["k"], alone["v"], o1, lse1, alone["do"])
    assert torch.equal(gr.dq[:, n - last:], gr1.dq)
    # dk and dv are sums of the same products in an order that goes by the call's size (which waves
    # share keys): fp32 sums of `last` terms in two orders differ by at most 2 gamma_last times the
    # sum of the absolute terms, and values that close round to bf16 at most a step (2^-7) apart
    hq, hk, hv, hdo = (alone[m][0].float().transpose(0, 1).contiguous() for m in ("q", "k", "v", "do"))
    sc = torch.bmm(hq, hk.transpose(1, 2).contiguous()) / D ** 0.5
    P = torch.softmax(sc.masked_fill(torch.ones(last, last, device=dev()).triu(1).bool(), -np.inf), -1)
    dP = torch.bmm(hdo, hv.transpose(1, 2).contiguous())
    dS = (P * (dP - (P * dP).sum(-1, keepdim=True))).abs() / D ** 0.5
    terms = {"dk": torch.bmm(dS.transpose(1, 2).contiguous(), hq.abs()),
             "dv": torch.bmm(P.transpose(1, 2).contiguous(), hdo.abs())}
    for name, t in terms.items():
        a, b = getattr(gr, name)[0, n - last:].float(), getattr(gr1, name)[0].float()
        # (1.01: the terms themselves are formed in fp32 here and from bf16 weights there)
        bound = 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 2 * gamma(last) * 1.01 * t.transpose(0, 1)
        assert ((a - b).abs() <= bound).all(), name
    del gr, o, lse
    torch.cuda.empty_cache()
    o, _ = pkv.chunk_linear_attn_varlen(x["q"], x["k"], x["v"], g, cu_gpu(cu), output_final_state=False)
    o1, _ = pkv.chunk_linear_attn_varlen(alone["q"], alone["k"], alone["v"], g, output_final_state=False)
    assert torch.equal(o[:, n - last:], o1)
    gr = pkv.chunk_linear_attn_varlen_backward(x["q"], x["k"], x["v"], g, x["do"], cu_gpu(cu))
    gr1 = pkv.chunk_linear_attn_varlen_backward(alone["q"], alone["k"], alone["v"], g, alone["do"])
    for a, b in zip(gr[:3], gr1[:3]):
        assert torch.equal(a[:, n - last:], b)
