"""What a mask hides weighs exactly 0, however large it is as long as it is finite."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu

HUGE = 3e38


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


CASES = [(300, 2, 1, 64, 60, 4), (300, 4, 2, 128, 60, 4), (400, 2, 2, 32, 100, 0), (2300, 1, 1, 64, 2200, 4)]


@pytest.mark.parametrize("T,Hq,Hkv,hd,window,n_sink", CASES)
def test_values_that_are_hidden(ttcd, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = (x.cuda() for x in make_attention_inputs(1, T, Hq, Hkv, hd, seed=T))
    o, lse = ttcd.sink_window_attn(q, k, v, window, n_sink, lse=True)
    for j in (*range(168, 176), T - 1):  # every column modulo 8
        w = v.clone()
        w[0, j] = HUGE
        o2, lse2 = ttcd.sink_window_attn(q, k, w, window, n_sink, lse=True)
        hid = torch.from_numpy(~so.mask(np.arange(T), [j], window, n_sink)[:, 0]).cuda()
        assert torch.equal(o2[0, hid], o[0, hid]) and torch.equal(lse2, lse)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("max_q", [1, 30])
def test_values_that_are_hidden_in_pages(ttcd, hd, max_q):
    """A chunk of 30 tokens: the later ones' values, and those that only the earlier see."""
    L, n, page, window, n_sink = 200, 30, 16, 50, 4
    g = torch.Generator().manual_seed(hd)
    kp, vp = (torch.randn(13, 1, page, hd, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(n, 2, hd, generator=g).bfloat16().cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda v: ttcd.paged_window_attn(q, kp, v, i32(*range(13)).view(1, 13), i32(0, n), i32(L),  # noqa: E731
                                            window, n_sink, max_q=max_q, lse=True)
    o, lse = call(vp)
    for j in (*range(L - 16, L), *range(L - n - window + 1, L - n - window + 17)):
        w = vp.clone()
        w[j // page, 0, j % page] = HUGE
        o2, lse2 = call(w)
        hid = torch.from_numpy(~so.mask(np.arange(L - n, L), [j], window, n_sink)[:, 0]).cuda()
        assert torch.equal(o2[hid], o[hid]) and torch.equal(lse2, lse)


@pytest.mark.parametrize("T,Hq,Hkv,hd,window,n_sink", [c for c in CASES if c[3] != 32])
def test_output_gradients_that_are_hidden(ttcd, T, Hq, Hkv, hd, window, n_sink):
    """dv of the keys that a query does not see has nothing of its output gradient."""
    q, k, v = (x.cuda() for x in make_attention_inputs(1, T, Hq, Hkv, hd, seed=T))
    d_o = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = ttcd.sink_window_attn(q, k, v, window, n_sink, lse=True)
    dv = ttcd.sink_window_attn_backward(q, k, v, o, lse, d_o, window, n_sink)[2]
    for t in (*range(164, 172), T - 70):
        big = d_o.clone()
        big[0, t] = HUGE
        got = ttcd.sink_window_attn_backward(q, k, v, o, lse, big, window, n_sink)[2]
        hid = torch.from_numpy(~so.mask([t], np.arange(T), window, n_sink)[0]).cuda()
        assert torch.equal(got[0, hid], dv[0, hid])
