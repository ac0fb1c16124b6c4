"""The softmax layer around the packed attention on the GPU against the fp64 oracle,
with the bounds of softmax_parity.py, and its invariants bit by bit."""

import numpy as np
import pytest
import torch

import packed_varlen_gated_amd as pkv
from mixer_parity import check
from oracle import mixers, softmax
from softmax_parity import norm_rope_bounds, paged_bounds, window_bounds
from test_gpu_mixers import DT, LENS, TAIL, attn_inputs, cu_gpu, dev, host, lay, on_gpu

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev())


def f32(a):
    return None if a is None else torch.from_numpy(np.asarray(a)).float().to(dev())


# ------------------------------------------------- norms and rotation

def rope_case(N, Hq, Hkv, D, dtype, rot=None, interleaved=False, weights=True, pos=None, fused=False, seed=0, eps=1e-6,
              amp=1.0):
    rng = np.random.default_rng(seed)
    rot = D if rot is None else rot
    freq = None if rot == 0 else (10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)
    w = {x: (1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if weights else None for x in "qk"}
    if fused:
        qkv = on_gpu(amp * rng.standard_normal((1, N, Hq + 2 * Hkv, D)), dtype)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    else:
        q, k = (on_gpu(amp * rng.standard_normal((1, N, h, D)), dtype) for h in (Hq, Hkv))
    dy = {x: on_gpu(rng.standard_normal((1, N, h, D)), dtype) for x, h in (("q", Hq), ("k", Hkv))}
    p = np.arange(N) if pos is None else np.asarray(pos)
    args = (f32(w["q"]), f32(w["k"]), None if pos is None else i32(pos), f32(freq), eps, interleaved)
    qo, ko = pkv.qk_norm_rope(q, k, *args)
    gr = pkv.qk_norm_rope_backward(q, k, dy["q"], dy["k"], *args)
    torch.cuda.synchronize()
    for x, t, y, dx, dw in (("q", q, qo, gr.dq, gr.dq_weight), ("k", k, ko, gr.dk, gr.dk_weight)):
        b = norm_rope_bounds(host(t)[0], host(dy[x])[0], None if w[x] is None else w[x].astype(np.float64), p,
                             None if freq is None else freq.astype(np.float64), float(np.float32(eps)), interleaved, dtype)
        check(host(y)[0], *b["y"], dtype, x)
        check(host(dx)[0], *b["dx"], dtype, "d" + x)
        if weights:
            check(host(dw), *b["dw"], "f32", "dw" + x)
        else:
            assert dw is None


ROPE_TYPES = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("dtype,D", ROPE_TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(dtype, D, interleaved):
    rope_case(1, 1, 1, D, dtype, interleaved=interleaved)
    rope_case(37, 5, 3, D, dtype, interleaved=interleaved, seed=1)
    rope_case(130, 9, 1, D, dtype, rot=16, interleaved=interleaved, seed=2, fused=True)
    rope_case(65, 17, 17, D, dtype, rot=D - 16, interleaved=interleaved, seed=3, weights=False)
    rope_case(50, 4, 2, D, dtype, rot=0, interleaved=interleaved, seed=4)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_norm_rope_many_tokens(dtype, D):
    """More tokens than the reverse pass has waves, and enough for one wave a token in the forward pass."""
    rope_case(9001, 3, 2, D, dtype, fused=True)


@pytest.mark.parametrize("dtype,D", ROPE_TYPES)
def test_norm_rope_positions(dtype, D):
    rng = np.random.default_rng(5)
    far = rng.integers(0, 1 << 20, 40)
    far[:4] = [2 ** 31 - 1, 0, 1 << 24, (1 << 24) + 1]
    rope_case(40, 3, 2, D, dtype, pos=far, seed=5)
    out = np.arange(40)
    out[[0, 7, 8, 39]] = [-1, -5, -(2 ** 31), -1]
    rope_case(40, 3, 2, D, dtype, pos=out, seed=6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_rope_small_and_large_values(dtype):
    rope_case(30, 2, 1, 64, dtype, amp=1e-12, eps=1e-6, seed=7)     # eps rules
    rope_case(30, 2, 1, 64, dtype, amp=1e15, eps=0.0, seed=8)       # squares near 2^100


def test_norm_rope_left_out_rows_may_hold_anything():
    """Padding of NaN and infinities gives zeros and reaches no weight's gradient."""
    q, k, dq, dk = attn_inputs(9, 50, 4, 2, 64, "bf16")[:2] + attn_inputs(10, 50, 4, 2, 64, "bf16")[:2]
    w, freq = torch.ones(64, device=dev()), torch.rand(32, device=dev())
    pos = torch.arange(50, dtype=torch.int32, device=dev())
    pos[33:] = -1
    ref = pkv.qk_norm_rope_backward(q, k, dq, dk, w, w, pos, freq)
    for t in (q, k, dq, dk):
        t[0, 33:40] = float("nan")
        t[0, 40:] = float("inf")
    got = pkv.qk_norm_rope_backward(q, k, dq, dk, w, w, pos, freq)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    y = pkv.qk_norm_rope(q, k, w, w, pos, freq)
    assert all(not t[0, 33:].any() and t[0, :33].any() for t in y)


def test_norm_rope_strided_equals_dense_and_batches_flatten():
    rng = np.random.default_rng(11)
    qkv = on_gpu(rng.standard_normal((3, 50, 12, 64)), "bf16")
    pos = i32(rng.integers(0, 99, (3, 50)))
    freq, w = f32(rng.random(16)), f32(rng.random(64))
    q, k = qkv[:, :, 2:8], qkv[:, :, 8:11]
    a = pkv.qk_norm_rope(q, k, w, w, pos, freq)
    b = pkv.qk_norm_rope(q.reshape(1, 150, 6, 64), k.reshape(1, 150, 3, 64), w, w, pos.view(-1), freq)
    assert all(torch.equal(x.view(-1), y.view(-1)) for x, y in zip(a, b))
    one = pkv.qk_norm_rope(q[1:2, 7:8], k[1:2, 7:8], w, w, pos[1, 7:8], freq)     # one token: any stride
    assert all(torch.equal(x[0, 0], y[1, 7]) for x, y in zip(one, a))


# --------------------------------------------------------- windows

def window_run(q, k, v, do, window, sinks, cud, scale=None):
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, lse = pkv.attn_window_varlen(q, k, v, window, sinks, cud, scale, flags=flags)
    gr = pkv.attn_window_varlen_backward(q, k, v, o, lse, do, window, sinks, cud, scale, flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    return dict(o=o, lse=lse, dq=gr.dq, dk=gr.dk, dv=gr.dv)


def window_case(lens, tail, Hq, Hkv, D, dtype, window, sinks, seed=0, scale=None, amp=1.0, none=False):
    N, cu = lay(lens, tail)
    q, k, v, do = attn_inputs(seed, N, Hq, Hkv, D, dtype, amp)
    got = window_run(q, k, v, do, window, sinks, None if none else cu_gpu(cu), scale)
    want = window_bounds(host(q)[0], host(k)[0], host(v)[0], host(do)[0], window, sinks, None if none else cu, scale,
                         dtype)
    end = int(cu[-1])
    for name, (ref, bound, extra) in want.items():
        x = host(got[name])
        if name == "lse":
            assert (x[:, end:] == -np.inf).all()
            check(x[:, :end], ref[:, :end], bound[:, :end], "f32", name)
        else:
            assert not x[0, end:].any(), name
            check(x[0], ref, bound, dtype, name, extra)


WIN_TYPES = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (32, 3), (64, 64), (100, 1), (129, 40), (4000, 2)])
@pytest.mark.parametrize("dtype,D", WIN_TYPES)
@pytest.mark.parametrize("case", list(LENS))
def test_window(case, dtype, D, window, sinks):
    window_case(LENS[case], TAIL[case], 4, 2, D, dtype, window, sinks, seed=window)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 1), (8, 2), (5, 5)])
@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_window_heads(Hq, Hkv, dtype, D):
    window_case([270, 130], 3, Hq, Hkv, D, dtype, 50, 5, seed=Hq)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_window_one_segment_and_scales(dtype, D):
    window_case([300], 0, 2, 1, D, dtype, 70, 3, none=True)
    window_case([300], 0, 2, 1, D, dtype, 70, 3, scale=-0.3)
    window_case([300], 0, 2, 1, D, dtype, 70, 3, scale=0.0)
    window_case([300, 90], 0, 2, 1, D, dtype, 33, 2, amp=4.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(200, 4), (640, 64), (48, 33), (777, 0)])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (12, 6), (50, 50)])
def test_window_many_tiles(Hq, Hkv, D, window, sinks):
    """Calls of 13, 78 and 650 work-groups of 128 keys: one, two or four waves to 32 keys."""
    window_case([900, 300, 2, 400], 7, Hq, Hkv, D, "bf16", window, sinks, seed=5)


@pytest.mark.parametrize("dtype,D", WIN_TYPES)
def test_a_window_of_all_tokens_is_attn_varlen(dtype, D):
    N, cu = lay([90, 60, 140], 10)
    q, k, v, do = attn_inputs(3, N, 4, 2, D, dtype)
    o, lse = pkv.attn_varlen(q, k, v, cu_gpu(cu))
    gr = pkv.attn_varlen_backward(q, k, v, o, lse, do, cu_gpu(cu))
    got = window_run(q, k, v, do, N, 0, cu_gpu(cu))
    for n, t in dict(o=o, lse=lse, dq=gr.dq, dk=gr.dk, dv=gr.dv).items():
        assert torch.equal(got[n], t), n
    # one that hides nothing, through the windowed kernels: the same sums
    close = window_run(q, k, v, do, 140, 0, cu_gpu(cu))
    assert torch.equal(close["o"], o) and torch.equal(close["lse"], lse) and torch.equal(close["dq"], gr.dq)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(40, 0), (40, 5), (130, 1)])
def test_window_hidden_values_reach_nothing(dtype, D, window, sinks):
    """NaN and infinities in tokens that a row does not see leave its bits; those it sees arrive."""
    N, cu = lay([600, 77], 9)
    q, k, v, do = attn_inputs(4, N, 4, 2, D, dtype)
    ref, rl = pkv.attn_window_varlen(q, k, v, window, sinks, cu_gpu(cu))
    t = torch.arange(N, device=dev())
    for bad in (float("nan"), float("inf"), -float("inf")):
        for at in (0, 3, 64, 200, 255, 599, 601, 680):
            for where in ("kv", "v"):
                k2, v2 = k.clone(), v.clone()
                if where == "kv":
                    k2[0, at] = bad
                v2[0, at] = bad
                o, lse = pkv.attn_window_varlen(q, k2, v2, window, sinks, cu_gpu(cu))
                a, e = (0, 600) if at < 600 else (600, 677)
                sees = (t >= at) & (t < e) & ((t - at < window) | (at - a < sinks))
                if at >= 677:
                    sees[:] = False
                assert torch.equal(o[0][~sees], ref[0][~sees]) and torch.equal(lse[:, ~sees], rl[:, ~sees]), (bad, at)
                if where == "v":
                    assert torch.equal(lse, rl)
                    want = torch.full_like(o[0][sees], bad)
                    assert torch.equal(torch.nan_to_num(o[0][sees].float(), 7.0, 8.0, 9.0),
                                       torch.nan_to_num(want.float(), 7.0, 8.0, 9.0)), (bad, at)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_window_segments_are_isolated(dtype, D):
    N, cu = lay([190, 160, 240], 40)
    q, k, v, do = attn_inputs(3, N, 4, 2, D, dtype)
    ref = window_run(q, k, v, do, 50, 3, cu_gpu(cu))
    for t in (q, k, v, do):
        t[0, 190:350] = float("nan")
        t[0, 220] = float("inf")
        t[0, 590:] = float("nan")
    got = window_run(q, k, v, do, 50, 3, cu_gpu(cu))
    for name in ref:
        for sl in (slice(0, 190), slice(350, 590)):
            x, y = (r[name][:, sl] if name == "lse" else r[name][0, sl] for r in (got, ref))
            assert torch.equal(x, y), name
    assert not got["o"][0, 590:].any() and not got["dv"][0, 590:].any()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_window_packed_equals_alone_and_repeats(dtype, D):
    N, cu = lay([200, 57, 700], 0)
    q, k, v, do = attn_inputs(7, N, 4, 2, D, dtype)
    a, b = (window_run(q, k, v, do, 45, 2, cu_gpu(cu)) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert torch.equal(pkv.attn_window_varlen(q, k, v, 45, 2, cu_gpu(cu), output_lse=False)[0], a["o"])
    for s, e in zip(cu[:-1], cu[1:]):
        one = window_run(*(t[:, s:e].contiguous() for t in (q, k, v, do)), 45, 2, None)
        for n in one:
            x = a[n][:, s:e] if n == "lse" else a[n][0, s:e]
            assert torch.equal(x, one[n] if n == "lse" else one[n][0]), n


@pytest.mark.parametrize("bad", [[1, 5, 20], [0, 30, 20], [0, 10, 50], [-3, 10, 20], [0, 100, 20]])
def test_window_bad_cu_seqlens_set_the_flag(bad):
    q, k, v, do = attn_inputs(8, 40, 2, 2, 64, "bf16")
    cu = cu_gpu(bad)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, lse = pkv.attn_window_varlen(q, k, v, 4, 2, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS
    flags.zero_()
    pkv.attn_window_varlen_backward(q, k, v, o, lse, do, 4, 2, cu, flags=flags)
    assert int(flags) == pkv.FLAG_BAD_CU_SEQLENS


def test_window_many_empty_slots():
    lens = [0] * 4500 + [170] + [0] * 300 + [133, 1] + [0] * 77
    window_case(lens, 5, 2, 1, 64, "bf16", 30, 2)
    window_case(lens, 5, 2, 1, 64, "bf16", 70, 2)


@pytest.mark.parametrize("D", [64, 128])
def test_window_short_segments_many_heads(D):
    rng = np.random.default_rng(17)
    lens = []
    while sum(lens) < 13300:
        lens.append(int(rng.integers(1, 260)))
    lens[3:3] = [0] * 600
    window_case(lens, 21, 10, 10, D, "bf16", 40, 3, seed=18)


# ------------------------------------------------------ the paged cache

def cache_of(rng, lens, size, Hkv, D, dtype, spare=3, fill=None):
    """(table, k_pages, v_pages) with the requests' pages in any order; what no token has is `fill` (or random)."""
    need = [-(-n // size) for n in lens]
    pages = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), 1 << 30)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = pages[at:at + n]
        at += n
    kp, vp = (rng.standard_normal((len(pages), size, Hkv, D)) for _ in range(2))
    if fill is not None:
        used = np.zeros((len(pages), size), dtype=bool)
        for r, n in enumerate(lens):
            used.reshape(-1)[softmax.places(table[r], n, size)] = True
        kp[~used], vp[~used] = fill, fill
    return table, on_gpu(kp, dtype), on_gpu(vp, dtype)


def paged_case(lens, news, Hq, Hkv, D, dtype, size, window=0, sinks=0, tail=0, seed=0, scale=None, amp=1.0,
               fill=float("nan"), one_each=False):
    """lens: the requests' tokens with the new ones; news: how many of them are new."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(news)])
    N = int(cu[-1]) + tail
    table, kp, vp = cache_of(rng, lens, size, Hkv, D, dtype, fill=fill)
    q = on_gpu(amp * rng.standard_normal((N, Hq, D)), dtype)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    o, lse = pkv.attn_paged(q, kp, vp, i32(table), i32(lens), None if one_each else i32(cu), window or None, sinks,
                            scale, output_lse=True, flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    clean = lambda x: np.nan_to_num(host(x), nan=0.0, posinf=0.0, neginf=0.0)
    want = paged_bounds(host(q), clean(kp), clean(vp), table, lens, cu, window, sinks, scale, dtype)
    ref, bound = want["lse"]
    got = host(lse)
    dead = np.isinf(ref)
    assert (got[dead] == -np.inf).all()
    check(np.where(dead, 0, got), np.where(dead, 0, ref), bound, "f32", "lse")
    check(host(o), *want["o"], dtype, "o")
    assert not host(o)[int(cu[-1]):].any()
    return o, lse


PAGED_TYPES = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]
DECODE = [1, 2, 16, 17, 0, 63, 64, 65, 300, 129, 0, 1000]


@pytest.mark.parametrize("size", [16, 48, 64, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 3), (100, 0), (130, 64)])
@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
def test_paged_one_token_each(dtype, D, window, sinks, size):
    paged_case(DECODE, [1] * len(DECODE), 4, 2, D, dtype, size, window, sinks, seed=size, one_each=True)


@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 0), (50, 2), (200, 33)])
@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
def test_paged_chunks(dtype, D, window, sinks):
    """Chunks and single tokens, requests without new tokens, a first chunk, rows that see nothing, a tail."""
    paged_case([500, 1, 40, 333, 0, 64, 200, 700], [130, 1, 40, 0, 3, 7, 1, 65], 4, 2, D, dtype, 16, window, sinks,
               tail=5, seed=window)
    paged_case([900], [310], 2, 1, D, dtype, 64, window, sinks, seed=window + 1)


@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
def test_paged_rows_before_the_first_place(dtype, D, window, sinks):
    """More new tokens than kv_lens: those before the first place see nothing."""
    paged_case([3, 0, 10, 200, 1, 0], [7, 4, 30, 300, 2, 150], 4, 2, D, dtype, 16, window, sinks, tail=2, seed=window)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 1), (8, 2), (5, 5), (40, 1), (16, 2), (140, 1)])
@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_paged_heads(Hq, Hkv, dtype, D):
    paged_case([270, 130, 31], [3, 1, 31], Hq, Hkv, D, dtype, 32, seed=Hq)
    paged_case([270, 130, 31], [1, 1, 1], Hq, Hkv, D, dtype, 32, 60, 4, seed=Hq, one_each=True)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_paged_scales(dtype, D):
    for kw in (dict(scale=-0.3), dict(scale=0.0), dict(amp=4.0)):
        paged_case([300, 90], [1, 1], 4, 2, D, dtype, 16, seed=2, **kw)
        paged_case([300, 90], [70, 33], 4, 2, D, dtype, 16, 40, 2, seed=3, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_paged_long_and_short_requests(D):
    """A walk of many work-groups beside short ones; more requests than a work-group has threads."""
    paged_case([5000, 3, 90, 0, 2500], [1, 1, 1, 1, 1], 8, 4, D, "bf16", 64, seed=1, one_each=True)
    paged_case([4000, 90, 2500], [200, 1, 33], 4, 2, D, "bf16", 16, seed=2)
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 700)
    lens[650] = 3000
    paged_case(lens.tolist(), [1] * 700, 4, 2, D, "bf16", 16, seed=4, one_each=True)
    news = np.minimum(lens, rng.integers(0, 20, 700))
    paged_case(lens.tolist(), news.tolist(), 4, 2, D, "bf16", 32, 50, 4, tail=3, seed=5)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1700, 40)])
@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32)])
def test_paged_long_walks_in_parts(dtype, D, window, sinks):
    """Few requests with long walks: many work-groups to each; a table far wider than its requests."""
    paged_case([9001], [1], 8, 2, D, dtype, 64, window, sinks, seed=1, one_each=True)
    paged_case([0, 4500, 3, 2049], [1, 1, 1, 1], 3, 1, D, dtype, 16, window, sinks, seed=2, one_each=True)
    paged_case([2600, 0, 40, 3100], [37, 1, 0, 9], 4, 2, D, dtype, 32, window, sinks, tail=3, seed=3)
    rng = np.random.default_rng(4)
    lens, cu = [2500, 900], np.array([0, 5, 6])
    table, kp, vp = cache_of(rng, lens, 16, 2, D, dtype)
    q = on_gpu(rng.standard_normal((6, 4, D)), dtype)
    wide = i32(np.concatenate([table, np.full((2, 4000), -1)], 1))
    b = paged_bounds(host(q), host(kp), host(vp), table, lens, cu, window, sinks, None, dtype)
    for t in (i32(table), wide):
        o, lse = pkv.attn_paged(q, kp, vp, t, i32(lens), i32(cu), window or None, sinks, output_lse=True)
        check(host(o), *b["o"], dtype, "o")
        check(host(lse), *b["lse"], "f32", "lse")
    # a value that is not finite reaches the rows that see it, whichever part has it
    for bad in (float("nan"), float("inf"), -float("inf")):
        for at in (0, 39, 41, 700, 1500, 2495, 2497, 2499):
            v2 = vp.clone()
            v2[int(table[0, at // 16]), at % 16] = bad
            got, l2 = pkv.attn_paged(q, kp, v2, wide, i32(lens), i32(cu), window or None, sinks, output_lse=True)
            see = softmax.visible(np.arange(2495, 2500), np.array([at]), window, sinks)[:, 0]
            sees = torch.from_numpy(np.append(see, False)).to(dev())
            assert torch.equal(got[~sees], o[~sees]) and torch.equal(l2, lse)
            want = torch.full_like(got[sees], bad).float()
            assert torch.equal(torch.nan_to_num(got[sees].float(), 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_paged_equals_packed(dtype, D):
    """A prompt's only chunk over the cache is the packed call's segment (up to the order of sums)."""
    N, cu = lay([200, 57, 300], 0)
    q, k, v, _ = attn_inputs(7, N, 4, 2, D, dtype)
    lens = np.diff(cu)
    rng = np.random.default_rng(1)
    table, kp, vp = cache_of(rng, lens.tolist(), 16, 2, D, dtype)
    pkv.paged_kv_append(k[0], v[0], kp, vp, i32(table), i32(lens), cu_gpu(cu))
    for window, sinks in ((0, 0), (70, 3)):
        o, lse = pkv.attn_paged(q[0], kp, vp, i32(table), i32(lens), cu_gpu(cu), window or None, sinks, output_lse=True)
        ro, rl = pkv.attn_window_varlen(q, k, v, window or N, sinks if window else 0, cu_gpu(cu))
        # two results within the same bounds of the same value
        b = paged_bounds(host(q)[0], host(kp), host(vp), table, lens, cu, window, sinks, None, dtype)
        assert (np.abs(host(o) - host(ro)[0]) <= 2 * b["o"][1]).all()
        assert (np.abs(host(lse) - host(rl)) <= 2 * b["lse"][1]).all()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 5)])
def test_paged_hidden_values_reach_nothing(dtype, D, window, sinks):
    """NaN and infinities in places that a row does not see leave its bits; a value that it sees arrives."""
    rng = np.random.default_rng(2)
    lens, news = [400, 90, 300, 30], [100, 1, 4, 30]
    cu = np.concatenate([[0], np.cumsum(news)])
    table, kp, vp = cache_of(rng, lens, 16, 2, D, dtype)
    q = on_gpu(rng.standard_normal((int(cu[-1]), 4, D)), dtype)
    call = lambda a, b: pkv.attn_paged(q, a, b, i32(table), i32(lens), i32(cu), window or None, sinks, output_lse=True)
    ref, rl = call(kp, vp)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for r, at in ((0, 0), (0, 4), (0, 299), (0, 333), (0, 399), (1, 50), (2, 2), (2, 260), (2, 298), (3, 11)):
            for where in ("kv", "v"):
                k2, v2 = kp.clone(), vp.clone()
                page, i = int(table[r, at // 16]), at % 16
                if where == "kv":
                    k2[page, i] = bad
                v2[page, i] = bad
                o, lse = call(k2, v2)
                sees = torch.zeros(len(q), dtype=torch.bool, device=dev())
                see = softmax.visible(np.arange(lens[r] - news[r], lens[r]), np.array([at]), window, sinks)[:, 0]
                sees[cu[r]:cu[r + 1]] = torch.from_numpy(see).to(dev())
                assert torch.equal(o[~sees], ref[~sees]) and torch.equal(lse[:, ~sees], rl[:, ~sees]), (bad, r, at)
                if where == "v":
                    assert torch.equal(lse, rl)
                    want = torch.full_like(o[sees], bad)
                    assert torch.equal(torch.nan_to_num(o[sees].float(), 7.0, 8.0, 9.0),
                                       torch.nan_to_num(want.float(), 7.0, 8.0, 9.0)), (bad, r, at)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_paged_bad_numbers_set_their_flags(dtype, D):
    """A bad length, page or cu_seqlens sets its flag; the other requests have their results, nothing else is written."""
    rng = np.random.default_rng(6)
    lens = [70, 40, 100]
    table, kp, vp = cache_of(rng, lens, 16, 2, D, dtype)
    q, k, v = (on_gpu(rng.standard_normal((3, h, D)), dtype) for h in (4, 2, 2))
    ref, _ = pkv.attn_paged(q, kp, vp, i32(table), i32(lens))
    # where a request's keys are cut goes by the lengths of the call's requests, and with it the order of its sums:
    # both results are within the bounds of the same value, so within twice that of each other
    bound = 2 * paged_bounds(host(q), host(kp), host(vp), table, lens, np.arange(4), 0, 0, None, dtype)["o"][1]
    same = lambda o: (np.abs(host(o) - host(ref)) <= bound)[[0, 2]].all()
    flags = torch.zeros(1, dtype=torch.int32, device=dev())

    def both(table, lens, cu=None):
        flags.zero_()
        o, _ = pkv.attn_paged(q, kp, vp, i32(table), i32(lens), cu, flags=flags)
        f = int(flags)
        flags.zero_()
        k2, v2 = kp.clone(), vp.clone()
        pkv.paged_kv_append(k, v, k2, v2, i32(table), i32(lens), cu, flags=flags)
        return o, f, int(flags), k2, v2
    for bad in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1):
        o, f, g, k2, v2 = both(table, [70, bad, 100])
        assert f == g == pkv.FLAG_BAD_LENGTH and same(o)
        changed = (k2 != kp).flatten(1).any(1).sum()
        assert int(changed) == 2
    for bad in (-1, len(kp), 2 ** 31 - 1, -(2 ** 31)):
        t = table.copy()
        t[1, 2] = bad                    # the page of request 1's last token
        o, f, g, k2, v2 = both(t, lens)
        assert f == g == pkv.FLAG_BAD_PAGE and torch.equal(o[[0, 2]], ref[[0, 2]])
        assert int((k2 != kp).flatten(1).any(1).sum()) == 2
    t = table.copy()
    t[1, 3] = -7                         # behind its last token: not needed
    o, f, g, _, _ = both(t, lens)
    assert f == g == 0 and torch.equal(o, ref)
    for cu in ([1, 1, 2, 3], [0, 2, 1, 3], [0, 1, 2, 9], [0, -1, 2, 3]):
        _, f, g, _, _ = both(table, lens, i32(cu))
        assert f == g == pkv.FLAG_BAD_CU_SEQLENS


@pytest.mark.parametrize("dtype,D", PAGED_TYPES)
@pytest.mark.parametrize("size", [16, 80, 256])
def test_append(dtype, D, size):
    rng = np.random.default_rng(size)
    for Hkv in (1, 2, 5):
        lens, news = [70, 1, 0, 333, 16, 40, 3], [70, 1, 2, 100, 0, 17, 5]   # request 2 idle, 6 longer than its cache
        cu = np.concatenate([[0], np.cumsum(news)])
        table, kp, vp = cache_of(rng, lens, size, Hkv, D, dtype)
        N = int(cu[-1]) + 4
        qkv = on_gpu(rng.standard_normal((N, 3 * Hkv, D)), dtype)
        k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        rk, rv = softmax.paged_kv_append(host(k), host(v), host(kp), host(vp), table, lens, cu)
        flags = torch.zeros(1, dtype=torch.int32, device=dev())
        k2, v2 = kp.clone(), vp.clone()
        pkv.paged_kv_append(k, v, k2, v2, i32(table), i32(lens), i32(cu), flags=flags)
        assert int(flags) == 0 and np.array_equal(host(k2), rk) and np.array_equal(host(v2), rv)
        one = [70, 1, 0, 333, 16, 40, 3]
        rk, rv = softmax.paged_kv_append(host(k)[:7], host(v)[:7], host(kp), host(vp), table, one)
        pkv.paged_kv_append(k[:7].contiguous(), v[:7], kp, vp, i32(table), i32(one))
        assert np.array_equal(host(kp), rk) and np.array_equal(host(vp), rv)


# ------------------------------------------------- used together, and how

@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (25, 3)])
def test_a_prompt_and_its_decoding(dtype, D, window, sinks):
    """Token rows -> positions and cu_seqlens -> norms and rotation -> attention, packed; then the same prompts
    in a cache, a chunk more and token by token, give what the longer packed prompts give."""
    rng = np.random.default_rng(11)
    Hq, Hkv, T, more = 4, 2, 150, 6
    tokens = rng.integers(1, 9, (1, T)).astype(np.int32)
    tokens[0, [40, 97, T - 1]] = 0
    seg = pkv.eod_to_segment_ids(torch.from_numpy(tokens).to(dev()), 0)
    cu = pkv.segment_ids_to_cu_seqlens(seg.segment_ids, 3).cu_seqlens
    starts = cu.cpu().numpy()
    w, freq = f32(1 + 0.2 * rng.standard_normal(D)), f32(100.0 ** (-np.arange(D // 2) * 2 / D))
    lens = np.diff(starts) + more
    longer = np.concatenate([[0], np.cumsum(lens)])
    full = on_gpu(rng.standard_normal((1, int(longer[-1]), Hq + 2 * Hkv, D)), dtype)
    idx = np.concatenate([longer[r] + np.arange(n) for r, n in enumerate(np.diff(starts))])

    def norm(x, pos):
        return pkv.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], w, w, pos, freq)
    at = lambda x: x[:, :, Hq + Hkv:].contiguous()
    win = (1 << 20, 0) if window is None else (window, sinks)
    # the prompts alone: packed, positions of the data pipeline
    x = full[:, idx].contiguous()
    q, k = norm(x, seg.positions)
    o, _ = pkv.attn_window_varlen(q, k, at(x), *win, cu)
    # the longer prompts, packed
    pos = np.concatenate([np.arange(n) for n in lens])
    fq, fk = norm(full, i32(pos))
    want, _ = pkv.attn_window_varlen(fq, fk, at(full), *win, cu_gpu(longer))
    assert torch.equal(fq[:, idx], q) and torch.equal(fk[:, idx], k)
    tol = 2.0 ** -7 if dtype == "bf16" else 1e-5
    close = lambda a, b: float((a.float() - b.float()).norm()) <= tol * float(b.float().norm())
    assert close(o[0], want[0, idx])
    # the cache: the prompts, a chunk of 3, then one token at a time
    table, kp, vp = cache_of(rng, lens.tolist(), 16, Hkv, D, dtype, fill=float("nan"))
    done = np.diff(starts)
    pkv.paged_kv_append(k[0], at(x)[0], kp, vp, i32(table), i32(done), cu)
    for step in (3, 1, 1, 1):
        new = np.concatenate([longer[r] + done[r] + np.arange(step) for r in range(3)])
        done = done + step
        c = i32(np.arange(4) * step) if step > 1 else None
        y = full[:, new].contiguous()
        sq, sk = norm(y, i32(pos[new]))
        pkv.paged_kv_append(sk[0], y[0, :, Hq + Hkv:], kp, vp, i32(table), i32(done), c)
        so, _ = pkv.attn_paged(sq[0], kp, vp, i32(table), i32(done), c, window, sinks)
        assert close(so, want[0, new]), step


def _layer(x):
    """Every call, as a training step and a decoding step make them."""
    args = (x["w"], x["w"], x["pos"], x["freq"])
    q, k = pkv.qk_norm_rope(x["q"], x["k"], *args)
    o, lse = pkv.attn_window_varlen(q, k, x["v"], 60, 3, x["cu"])
    ga = pkv.attn_window_varlen_backward(q, k, x["v"], o, lse, x["do"], 60, 3, x["cu"])
    gr = pkv.qk_norm_rope_backward(x["q"], x["k"], ga.dq, ga.dk, *args)
    pkv.paged_kv_append(k[0], x["v"][0], x["kp"], x["vp"], x["table"], x["lens"], x["cu"])
    po, pl = pkv.attn_paged(q[0], x["kp"], x["vp"], x["table"], x["lens"], x["cu"], output_lse=True)
    n = len(x["lens"])
    pd, _ = pkv.attn_paged(q[0, :n], x["kp"], x["vp"], x["table"], x["lens"], None, 60, 3)
    return [q, k, o, lse, *ga, *gr, x["kp"].clone(), x["vp"].clone(), po, pl, pd]


def _layer_inputs(dtype, D, seed):
    lens = [300, 40, 700]
    N, cu = lay(lens, 8)
    rng = np.random.default_rng(seed)
    q, k, v, do = attn_inputs(seed, N, 4, 2, D, dtype)
    table, kp, vp = cache_of(rng, lens, 16, 2, D, dtype)
    return dict(q=q, k=k, v=v, do=do, cu=cu_gpu(cu), pos=i32(rng.integers(0, 5000, N)), freq=f32(rng.random(D // 2)),
                w=f32(1 + rng.random(D)), table=i32(table), lens=i32(lens), kp=kp, vp=vp)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_captured_and_replayed(dtype, D):
    """Two captured graphs, replayed in turn with new inputs and eager work between, give the eager bits."""
    x = _layer_inputs(dtype, D, 21)
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(x)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _layer(x)
        graphs.append((g, outs))
    for i in range(5):
        new = _layer_inputs(dtype, D, 30 + i)
        for n in x:
            x[n].copy_(new[n])
        want = [t.clone() for t in _layer(x)]
        for n in ("kp", "vp"):
            x[n].copy_(new[n])
        g, outs = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (i, j)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_paged_captured_with_changing_lengths(dtype, D):
    """A captured call goes by the lengths, pages and chunks that the tensors hold at the replay."""
    rng = np.random.default_rng(5)
    lens = [900, 500, 1200, 64]
    table, kp, vp = cache_of(rng, lens, 16, 2, D, dtype)
    q = on_gpu(rng.standard_normal((160, 8, D)), dtype)
    lays = [([900, 500, 1200, 64], [0, 1, 2, 3, 4]), ([300, 2, 1100, 0], [0, 100, 102, 160, 160]),
            ([16, 17, 1200, 1], [0, 1, 17, 150, 151])]
    t, n, c = i32(table), i32(lays[0][0]), i32(lays[0][1])
    call = lambda: pkv.attn_paged(q, kp, vp, t, n, c, output_lse=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = call()
    for i in (0, 1, 2, 1, 0):
        n.copy_(i32(lays[i][0]))
        c.copy_(i32(lays[i][1]))
        want = [x.clone() for x in call()]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), i


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 128)])
def test_decoding_step_captured(dtype, D):
    """A step's append and attention, captured once: the caller's lengths grow by one between replays, over a page's end."""
    rng = np.random.default_rng(9)
    lens, steps = [300, 15, 1, 2000, 63], 5
    table, kp, vp = cache_of(rng, [n + steps + 1 for n in lens], 16, 2, D, dtype)
    q = on_gpu(rng.standard_normal((steps, 5, 8, D)), dtype)
    k, v = (on_gpu(rng.standard_normal((steps, 5, 2, D)), dtype) for _ in range(2))
    t, n = i32(table), i32(lens)

    def step(q, k, v, kp, vp):
        pkv.paged_kv_append(k, v, kp, vp, t, n)
        return pkv.attn_paged(q, kp, vp, t, n, output_lse=True)
    now = [x[0].clone() for x in (q, k, v)]
    pages = [kp.clone(), vp.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*now, kp.clone(), vp.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = step(*now, kp, vp)
    for i in range(steps):
        n += 1
        for x, y in zip(now, (q, k, v)):
            x.copy_(y[i])
        g.replay()
        want = step(q[i], k[i], v[i], *pages)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), i
        assert torch.equal(kp.nan_to_num(7.0), pages[0].nan_to_num(7.0)), i


def test_on_another_stream():
    x = _layer_inputs("bf16", 64, 40)
    y = {n: t.clone() for n, t in x.items()}
    want = _layer(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _layer(y)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 32)])
def test_two_calls_at_once(dtype, D):
    """Calls of two streams, each with its own workspace, do not disturb each other."""
    x, y = _layer_inputs(dtype, D, 41), _layer_inputs(dtype, D, 42)
    again = [{n: t.clone() for n, t in z.items()} for z in (x, y)]
    want = [_layer(x), _layer(y)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, z in zip(streams, again):
        with torch.cuda.stream(s):
            got.append(_layer(z))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_a_caller_s_workspace():
    x = _layer_inputs("bf16", 64, 43)
    N = x["q"].shape[1]
    o, lse = pkv.attn_window_varlen(x["q"], x["k"], x["v"], 60, 3, x["cu"])
    want = pkv.attn_window_varlen_backward(x["q"], x["k"], x["v"], o, lse, x["do"], 60, 3, x["cu"])
    for wrap in (lambda n: torch.full((n,), 255, dtype=torch.uint8, device=dev()),):
        ws = wrap(pkv.attn_window_varlen_backward_workspace_size(N, 4, 2, 64, 3, torch.bfloat16, 60, 3))
        got = pkv.attn_window_varlen_backward(x["q"], x["k"], x["v"], o, lse, x["do"], 60, 3, x["cu"], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        a = (x["q"], x["k"], x["do"], o[:, :, :2].contiguous(), x["w"], x["w"], x["pos"], x["freq"])
        ws = wrap(pkv.qk_norm_rope_backward_workspace_size(N, 4, 2, 64, torch.bfloat16))
        assert all(torch.equal(p, q) for p, q in zip(pkv.qk_norm_rope_backward(*a, workspace=ws),
                                                      pkv.qk_norm_rope_backward(*a)))
        with pytest.raises(ValueError, match="workspace holds"):
            pkv.qk_norm_rope_backward(*a, workspace=ws[:-1])
        need = pkv.attn_paged_workspace_size(N, 3, 4, 2, 64, torch.bfloat16)
        p = (x["q"][0], x["kp"], x["vp"], x["table"], x["lens"], x["cu"])
        if need:
            assert torch.equal(pkv.attn_paged(*p, workspace=wrap(need))[0], pkv.attn_paged(*p)[0])


def test_offsets_past_32_bits():
    """A cache and packed tensors of more than 2^31 elements: what lies at their ends equals the same alone."""
    D, Hkv, size = 128, 8, 64
    pages = (1 << 31) // (size * Hkv * D) + 40
    gen = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = (torch.empty(pages, size, Hkv, D, dtype=torch.bfloat16, device=dev()).normal_(generator=gen) for _ in range(2))
    assert kp.numel() > 1 << 31
    table = torch.arange(pages - 20, pages, dtype=torch.int32, device=dev()).view(2, 10).contiguous()
    lens = i32([640, 333])
    q = torch.randn(2, 32, D, device=dev(), generator=gen).bfloat16()
    k, v = (torch.randn(2, Hkv, D, device=dev(), generator=gen).bfloat16() for _ in range(2))
    small = [t[pages - 20:].clone() for t in (kp, vp)]
    near = (table - (pages - 20)).contiguous()
    for c, t in (((kp, vp), table), (small, near)):
        pkv.paged_kv_append(k, v, *c, t, lens)
    assert torch.equal(kp[pages - 20:], small[0]) and torch.equal(vp[pages - 20:], small[1])
    assert torch.equal(pkv.attn_paged(q, kp, vp, table, lens)[0], pkv.attn_paged(q, *small, near, lens)[0])
    assert torch.equal(pkv.attn_paged(q, kp, vp, table, lens, i32([0, 1, 2]))[0],
                       pkv.attn_paged(q, *small, near, lens, i32([0, 1, 2]))[0])
    del kp, vp
    torch.cuda.empty_cache()
    H, n, last = 128, 131400, 150
    x = {m: torch.empty(1, n, H, D, dtype=torch.bfloat16, device=dev()).normal_(generator=gen) for m in ("q", "k", "do")}
    w, freq = torch.ones(D, device=dev()), torch.rand(D // 2, device=dev(), generator=gen)
    pos = torch.arange(n, dtype=torch.int32, device=dev())
    end = {m: t[:, n - last:].contiguous() for m, t in x.items()}
    a = pkv.qk_norm_rope(x["q"], x["k"], w, w, pos, freq)
    b = pkv.qk_norm_rope(end["q"], end["k"], w, w, pos[n - last:], freq)
    assert all(torch.equal(s[:, n - last:], t) for s, t in zip(a, b))
    del a
    a = pkv.qk_norm_rope_backward(x["q"], x["k"], x["do"], x["do"], w, w, pos, freq)
    b = pkv.qk_norm_rope_backward(end["q"], end["k"], end["do"], end["do"], w, w, pos[n - last:], freq)
    assert all(torch.equal(s[:, n - last:], t) for s, t in zip(a[:2], b[:2]))
    del a
    torch.cuda.empty_cache()
    cu = torch.unique(torch.arange(n - last, dtype=torch.int64) // 137 * 137).tolist() + [n - last, n]
    o, lse = pkv.attn_window_varlen(x["q"], x["k"], x["do"], 70, 2, cu_gpu(cu))
    o1, lse1 = pkv.attn_window_varlen(end["q"], end["k"], end["do"], 70, 2)
    assert torch.equal(o[:, n - last:], o1) and torch.equal(lse[:, n - last:], lse1)
    gr = pkv.attn_window_varlen_backward(x["q"], x["k"], x["do"], o, lse, x["q"], 70, 2, cu_gpu(cu))
    gr1 = pkv.attn_window_varlen_backward(end["q"], end["k"], end["do"], o1, lse1, end["q"], 70, 2)
    assert torch.equal(gr.dq[:, n - last:], gr1.dq)
    # dk and dv are sums of the same products in an order that goes by the call's size (which waves share
    # keys): both lie within the bounds around the oracle's
    want = window_bounds(*(host(end[m])[0] for m in ("q", "k", "do", "q")), 70, 2, None, None, "bf16")
    for name, got in (("dk", gr.dk[0, n - last:]), ("dv", gr.dv[0, n - last:]), ("dk", gr1.dk[0]), ("dv", gr1.dv[0])):
        check(host(got), *want[name][:2], "bf16", name, want[name][2])
