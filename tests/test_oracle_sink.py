"""The float64 oracle of sliding-window attention with sinks, pinned: against
torch's softmax and autograd in float64, against differences, and against the
windowed oracle where there are no sinks."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from oracle import ttcd_oracle as orc

CASES = [  # B, T, Hq, Hkv, hd, window, n_sink
    (2, 37, 4, 2, 8, 5, 3),
    (1, 20, 3, 1, 4, 1, 0),
    (1, 33, 2, 2, 8, 64, 4),   # window longer than the sequence
    (1, 16, 2, 1, 4, 3, 16),   # every key is a sink: causal
    (1, 1, 1, 1, 4, 1, 1),
]


def _inputs(B, T, Hq, Hkv, hd, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, T, Hq, hd)), r.standard_normal((B, T, Hkv, hd)),
            r.standard_normal((B, T, Hkv, hd)), r.standard_normal((B, T, Hq, hd)))


def _torch(q, k, v, window, n_sink, scale):
    T, G = q.shape[1], q.shape[2] // k.shape[2]
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bthd,bjhd->bhtj", q, k) * scale
    t = torch.arange(T)
    hide = torch.tensor([[not (j <= i and (i - j < window or j < n_sink)) for j in range(T)]
                         for i in range(T)])
    s = s.masked_fill(hide, float("-inf"))
    return torch.einsum("bhtj,bjhd->bthd", torch.softmax(s, -1), v), torch.logsumexp(s, -1)


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", CASES)
def test_against_torch(B, T, Hq, Hkv, hd, window, n_sink):
    x = _inputs(B, T, Hq, Hkv, hd)
    q, k, v, d_o = (torch.from_numpy(a).requires_grad_(i < 3) for i, a in enumerate(x))
    o, lse = _torch(q, k, v, window, n_sink, 0.3)
    ro, rl, _ = so.sink_window_attention(*x[:3], window, n_sink, 0.3)
    np.testing.assert_allclose(ro, o.detach(), atol=1e-12)
    np.testing.assert_allclose(rl, lse.detach(), atol=1e-12)
    g, _ = so.sink_window_attention_vjp(*x, window, n_sink, 0.3)
    for a, b in zip(torch.autograd.grad(o, (q, k, v), d_o), (g["dq"], g["dk"], g["dv"])):
        np.testing.assert_allclose(b, a, atol=1e-12)


def test_gradient_against_differences():
    x = _inputs(1, 11, 2, 1, 4, seed=3)
    g, _ = so.sink_window_attention_vjp(*x, 3, 2, 0.5)
    r = np.random.default_rng(4)
    for i, n in enumerate(("dq", "dk", "dv")):
        d = r.standard_normal(x[i].shape)
        h = 1e-5
        up, dn = ([a + s * h * d if j == i else a for j, a in enumerate(x[:3])] for s in (1, -1))
        f = [(so.sink_window_attention(*y, 3, 2, 0.5)[0] * x[3]).sum() for y in (up, dn)]
        assert abs((f[0] - f[1]) / (2 * h) - (g[n] * d).sum()) < 1e-7


def test_without_sinks_it_is_the_window():
    q, k, v, _ = _inputs(2, 50, 4, 2, 8, seed=1)
    o, lse, _ = so.sink_window_attention(q, k, v, 7, 0, 0.4)
    oT, _, lT, _ = orc.dual_window_attention(q, k, v, 7, 7, 0.4)
    np.testing.assert_allclose(o, oT, atol=1e-12)
    np.testing.assert_allclose(lse, lT, atol=1e-12)


def test_rotation_is_a_rotation_by_the_position():
    r = np.random.default_rng(2)
    x = r.standard_normal((5, 3, 8))
    np.testing.assert_allclose(so.rotate(x, np.zeros(5), 100.0), x, atol=1e-15)
    a, b = so.rotate(x, [3, 4, 5, 6, 7], 100.0), so.rotate(x, [13, 14, 15, 16, 17], 100.0)
    # inner products depend on the difference of positions only
    np.testing.assert_allclose((a[0] * a[2]).sum(-1), (b[0] * b[2]).sum(-1), atol=1e-12)
    np.testing.assert_allclose(a[0, 0, 0], x[0, 0, 0] * np.cos(3) - x[0, 0, 4] * np.sin(3))
    np.testing.assert_allclose(a[0, 0, 7], x[0, 0, 7] * np.cos(3 * 100 ** -0.75) +
                               x[0, 0, 3] * np.sin(3 * 100 ** -0.75))
