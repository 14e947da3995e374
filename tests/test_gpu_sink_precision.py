"""What the sink-window kernels keep beside the bounds of bf16 operands: gradients of a
sink without a second rounding, the log-sum-exp in 32-bit quality, and the bits of
every run."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests import coherent_sink as cs
from tests.helpers import np64
from tests.test_gpu_sink_attention import _within
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


@pytest.mark.parametrize("hd,T,Hq,seed", cs.CASES)
def test_gradients_of_a_sink_are_rounded_once(ttcd, hd, T, Hq, seed):
    """tests/test_coherent_sink.py shows that P or dS as one bf16 for the sink, or delta
    from the rounded o, would break these bounds."""
    x = cs.inputs(hd, T, Hq, seed)
    q, k, v, d_o = (y.cuda() for y in x)
    o, lse = ttcd.sink_window_attn(q, k, v, cs.WINDOW, 1, lse=True)
    dq, dk, dv, ws = ttcd.sink_window_attn_backward(q, k, v, o, lse, d_o, cs.WINDOW, 1)
    assert ttcd.check_device_status(ws) == ttcd.OK
    ref, bound = cs.exact(*x)
    _within(dq[0], ref["dq"], bound["dq"], "dq")
    _within(dk[0, 0, 0], ref["dk"], bound["dk"], "dk")
    _within(dv[0, 0, 0], ref["dv"], bound["dv"], "dv")


@pytest.mark.parametrize("hd", [32, 64, 128])
def test_lse_keeps_32_bit_quality(ttcd, hd):
    """Almost all weight on keys whose exponentials the tiled kernel forms on the FMA pipe
    (columns 6 and 7 modulo 8), where a cubic has an error of nearly 1e-4 of one sign.

    Bound: 2.8e-6 of the quartic; 16 additions in each of 8 chains and 3 to join them,
    per visit, 2^-24 each and two visits at most: 2.3e-6; 2^-22 of a hardware
    exponential; two ulps of the hardware logarithm (below 8): 2^-20 ln 2; a few 2^-24 of
    scores and sums below 8: 2^-21.  Together 6.5e-6."""
    T, y = 256, -0.34375  # the exponent: near the largest error of the cubic, 1.0e-4
    scale = float(np.float32(np.log(2)))
    q = torch.zeros(1, T, 2, hd, dtype=torch.bfloat16)
    q[..., 0] = 1
    k, v = torch.zeros(1, T, 1, hd, dtype=torch.bfloat16), torch.randn(1, T, 1, hd).bfloat16()
    at = torch.arange(T)
    k[0, :, 0, 0] = torch.where(at % 8 >= 6, y, torch.where(at % 64 == 0, 0.0, -40.0)).bfloat16()
    rl = np.stack([so.attend(np64(q)[0, :, h], np64(k)[0, :, 0], np64(v)[0, :, 0], at.numpy(),
                             at.numpy(), 1000, 0, scale)[1] for h in range(2)])
    _, lse = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), 1000, 0, scale=scale, lse=True)
    off = np.abs(np64(lse)[0] - rl)
    assert off.max() <= 6.5e-6, (off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("T,Hq,Hkv,hd,window,n_sink", [(900, 4, 2, 64, 100, 4), (700, 6, 2, 128, 700, 0)])
def test_gradients_repeat_their_bits_on_streams_and_in_graphs(ttcd, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = (x.cuda() for x in make_attention_inputs(2, T, Hq, Hkv, hd, seed=3))
    d_o = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()

    def step(stream=None):
        o, lse = ttcd.sink_window_attn(q, k, v, window, n_sink, lse=True, stream=stream)
        return (o, lse) + ttcd.sink_window_attn_backward(q, k, v, o, lse, d_o, window, n_sink,
                                                         stream=stream)[:3]

    want = step()
    torch.cuda.synchronize()
    for got in [step(torch.cuda.Stream()) for _ in range(4)]:  # side by side
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (4, 5):
        for x, y in zip((q, k, v), make_attention_inputs(2, T, Hq, Hkv, hd, seed=seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
