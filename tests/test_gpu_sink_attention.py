"""ttcd_sink_window_attn and its backward against the float64 oracle, element by
element within the bounds that the oracle derives from the roundings (half a step
of bf16 for P, dS and each output, 32-bit work on the rest)."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


def _inputs(B, T, Hq, Hkv, hd, seed):
    q, k, v = make_attention_inputs(B, T, Hq, Hkv, hd, seed=seed)
    assert so.score_slack(np64(q), np64(k), hd ** -0.5) <= 0.8 * so.W
    return q, k, v


def _within(got, ref, bound, what):
    got = np64(got)
    off = np.abs(got - ref)
    bad = ~(off <= bound + 1e-9)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float((off / (bound + 1e-9)).max()),
                           np.argwhere(bad)[:5].tolist())


CASES = [
    # B, T, Hq, Hkv, hd, window, n_sink
    (1, 1, 2, 1, 64, 4, 4),          # one token
    (1, 2, 4, 4, 128, 1, 0),         # two tokens, each sees itself
    (2, 300, 4, 2, 64, 48, 4),       # ragged length
    (1, 127, 2, 2, 128, 300, 1),     # a window beyond the sequence, no grouping
    (1, 129, 8, 1, 128, 128, 128),   # a tile and a token, a tile of sinks
    (2, 700, 6, 2, 64, 130, 7),      # groups of 3: 42 tokens a tile
    (1, 1000, 4, 2, 128, 100, 16),
    (1, 513, 5, 1, 32, 200, 3),      # head_dim 32, groups of 5
    (1, 640, 16, 1, 64, 33, 100),    # groups of 16, more sinks than window
    (1, 260, 128, 1, 64, 65, 2),     # groups of 128: one token a tile
    (3, 385, 2, 1, 128, 1, 1),       # itself and the first token
    (1, 1500, 4, 2, 64, 512, 0),     # no sinks
]


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", CASES)
def test_forward(ttcd, B, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T + hd)
    o, lse = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), window, n_sink, lse=True)
    torch.cuda.synchronize()
    assert ttcd.get_device_error()[0] == ttcd.OK
    ro, rl, bo = so.sink_window_attention(np64(q), np64(k), np64(v), window, n_sink, hd ** -0.5)
    _within(o, ro, bo, "o")
    # log of a sum of weights that are each off by W at most
    _within(lse, rl, so.W + 2.0 ** -22 * np.abs(rl), "lse")


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", [c for c in CASES if c[4] != 32])
def test_backward(ttcd, B, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T + hd + 1)
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=7)[0]
    qc, kc, vc = q.cuda(), k.cuda(), v.cuda()
    o, lse = ttcd.sink_window_attn(qc, kc, vc, window, n_sink, lse=True)
    dq, dk, dv, ws = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, d_o.cuda(), window, n_sink)
    torch.cuda.synchronize()
    assert ttcd.check_device_status(ws) == ttcd.OK
    g, e = so.sink_window_attention_vjp(np64(q), np64(k), np64(v), np64(d_o), window, n_sink,
                                        hd ** -0.5)
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        _within(x, g[n], e[n], n)


def test_gradient_against_differences(ttcd):
    """The directional derivative of sum(o d_o), in fp64 from the oracle's forward
    (differences of the bf16 kernel itself would be rounding noise)."""
    B, T, Hq, Hkv, hd, window, n_sink = 1, 150, 2, 1, 64, 40, 3
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=5)
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=8)[0]
    o, lse = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), window, n_sink, lse=True)
    got = ttcd.sink_window_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, d_o.cuda(), window,
                                         n_sink)
    x = [np64(q), np64(k), np64(v)]
    _, e = so.sink_window_attention_vjp(*x, np64(d_o), window, n_sink, hd ** -0.5)
    r = np.random.default_rng(0)
    for i, n in enumerate(("dq", "dk", "dv")):
        d, h = r.standard_normal(x[i].shape), 1e-4
        f = [(so.sink_window_attention(*[a + s * h * d if j == i else a for j, a in enumerate(x)],
                                       window, n_sink, hd ** -0.5)[0] * np64(d_o)).sum()
             for s in (1, -1)]
        # the bound of every element, and the third-order term of the differences
        tol = (e[n] * np.abs(d)).sum() + 1e-5
        assert abs((f[0] - f[1]) / (2 * h) - (np64(got[i]) * d).sum()) <= tol


@pytest.mark.parametrize("window,n_sink", [(1, 0), (16, 4), (100, 128), (128, 1), (300, 64)])
def test_mask_counts_are_exact(ttcd, window, n_sink):
    """Q = 0: every visible key has weight 1, so e^lse counts them."""
    T, hd = 600, 64
    q = torch.zeros(1, T, 2, hd, dtype=torch.bfloat16, device="cuda")
    _, k, v = make_attention_inputs(1, T, 1, 1, hd, seed=1)
    _, lse = ttcd.sink_window_attn(q, k.cuda(), v.cuda(), window, n_sink, lse=True)
    t = np.arange(T)
    want = so.mask(t, t, window, n_sink).sum(1)
    np.testing.assert_array_equal(np.rint(np.exp(np64(lse)[0, 0])), want)
    np.testing.assert_array_equal(np.rint(np.exp(np64(lse)[0, 1])), want)


def test_large_scores_stay_finite(ttcd):
    """Scores of hundreds, growing along the sequence: the running maximum moves
    many times.  The output is the value of the largest score."""
    T, hd = 500, 64
    q = torch.ones(1, T, 1, hd, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(T, device="cuda").view(1, T, 1, 1) * 1.0).expand(1, T, 1, hd).bfloat16().contiguous()
    v = torch.randn(1, T, 1, hd, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    o, lse = ttcd.sink_window_attn(q, k, v, 200, 4, lse=True)
    ro, rl, bo = so.sink_window_attention(np64(q), np64(k), np64(v), 200, 4, hd ** -0.5)
    # scores up to 4000 are exact sums here (whole numbers times 64 / 8)
    _within(o, ro, bo, "o")
    _within(lse, rl, 2.0 ** -20 * np.abs(rl) + 1e-4, "lse")
    assert torch.isfinite(o).all()


def test_sequences_do_not_see_each_other(ttcd):
    """NaN in one sequence of a batch does not reach the next."""
    q, k, v = (x.cuda() for x in make_attention_inputs(3, 200, 4, 2, 64, seed=2))
    o, lse = ttcd.sink_window_attn(q, k, v, 64, 4, lse=True)
    for x in (q, k, v):
        x[1] = float("nan")
    o2, lse2 = ttcd.sink_window_attn(q, k, v, 64, 4, lse=True)
    for b in (0, 2):
        assert torch.equal(o[b], o2[b]) and torch.equal(lse[b], lse2[b])
    assert torch.isnan(o2[1]).all()
    d_o = torch.ones_like(o)
    d_o[1] = float("nan")
    g = ttcd.sink_window_attn_backward(q, k, v, o2, lse2, d_o, 64, 4)
    for x in g[:3]:
        assert torch.isfinite(x[0]).all() and torch.isfinite(x[2]).all()


def test_streams_graphs_and_given_outputs(ttcd):
    q, k, v = (x.cuda() for x in make_attention_inputs(2, 400, 4, 2, 64, seed=3))
    d_o = torch.randn_like(q)
    o, lse = ttcd.sink_window_attn(q, k, v, 100, 4, lse=True)
    g = ttcd.sink_window_attn_backward(q, k, v, o, lse, d_o, 100, 4)
    out = torch.full_like(q, float("nan"))
    o1, none = ttcd.sink_window_attn(q, k, v, 100, 4, o=out)
    assert o1 is out and none is None and torch.equal(out, o)
    # on a stream of its own, twice at once
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a = ttcd.sink_window_attn(q, k, v, 100, 4, lse=True, stream=s1)
    b = ttcd.sink_window_attn(q, k, v, 100, 4, lse=True, stream=s2)
    ga = ttcd.sink_window_attn_backward(q, k, v, *a, d_o, 100, 4, stream=s1)
    gb = ttcd.sink_window_attn_backward(q, k, v, *b, d_o, 100, 4, stream=s2)
    torch.cuda.synchronize()
    for x in (a, b):
        assert torch.equal(x[0], o) and torch.equal(x[1], lse)
    for x in (ga, gb):
        for i in range(3):
            torch.testing.assert_close(x[i], g[i], rtol=2.0 ** -7, atol=1e-4)
    # captured, and replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, glse = ttcd.sink_window_attn(q, k, v, 100, 4, lse=True)
        gg = ttcd.sink_window_attn_backward(q, k, v, go, glse, d_o, 100, 4)
    for seed in (4, 5):
        for x, y in zip((q, k, v), make_attention_inputs(2, 400, 4, 2, 64, seed=seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = ttcd.sink_window_attn(q, k, v, 100, 4, lse=True)
        g2 = ttcd.sink_window_attn_backward(q, k, v, o2, lse2, d_o, 100, 4)
        assert torch.equal(go, o2) and torch.equal(glse, lse2)
        for i in range(3):
            torch.testing.assert_close(gg[i], g2[i], rtol=2.0 ** -7, atol=1e-4)


def test_refuses_what_it_cannot_take(ttcd):
    q, k, v = (x.cuda() for x in make_attention_inputs(1, 64, 4, 2, 64, seed=1))
    with pytest.raises(ValueError):
        ttcd.sink_window_attn(q, k[:, :32], v, 10, 1)
    with pytest.raises(ValueError):
        ttcd.sink_window_attn(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 10, 1)
    with pytest.raises(ttcd.TTCDError):
        ttcd.sink_window_attn(q.float(), k.float(), v.float(), 10, 1)
    with pytest.raises(ttcd.TTCDError):
        ttcd.sink_window_attn(q, k, v, 10, 129)
