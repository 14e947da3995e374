"""Scores that are not finite reach the result as they do in the formulas, whichever
column of a tile they are in and whichever kernel reads them: NaN and +inf make a
row NaN, -inf takes a key out of it.  Rows whose mask hides such a key do not see it."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from tests.test_gpu_sink_attention import _within
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


def _compare(got_o, got_lse, q, k, v, t, window, n_sink, what):
    """o [n, Hq, hd] and lse [Hq, n] against the oracle, which follows IEEE arithmetic."""
    Hq, hd = q.shape[1:]
    G = Hq // k.shape[1]
    for h in range(Hq):
        with np.errstate(invalid="ignore"):
            ro, rl, _, bo = so.attend(np64(q[:, h]), np64(k[:, h // G]), np64(v[:, h // G]), t,
                                      np.arange(len(k)), window, n_sink, hd ** -0.5)
        o, lse = np64(got_o[:, h]), np64(got_lse[h])
        lost = np.isnan(ro).any(-1)
        assert (np.isnan(ro).all(-1) == lost).all()
        np.testing.assert_array_equal(np.isnan(o), np.isnan(ro), err_msg=str((what, h)))
        np.testing.assert_array_equal(np.isnan(lse), np.isnan(rl), err_msg=str((what, h)))
        _within(o[~lost], ro[~lost], bo[~lost], (what, h))
        fine = np.isfinite(rl)
        _within(lse[fine], rl[fine], so.W + 2.0 ** -22 * np.abs(rl[fine]), (what, "lse", h))
        # a row without any score has the log of nothing
        np.testing.assert_array_equal(lse[np.isinf(rl)], rl[np.isinf(rl)])


def _key(k, j, kind):
    if kind == "nan":
        k[j] = NAN
    else:  # the sign of the query's first element decides between +inf and -inf
        k[j, :, 0] = INF


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("T,Hq,Hkv,hd,window,n_sink", [
    (400, 4, 2, 64, 100, 4),
    (400, 4, 2, 128, 100, 4),
    (300, 2, 1, 32, 300, 0),
    (2300, 1, 1, 64, 2200, 4),    # keys split over a cluster
    (2300, 3, 1, 128, 2200, 4),
])
def test_dense(ttcd, kind, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = make_attention_inputs(1, T, Hq, Hkv, hd, seed=T + hd)
    assert so.score_slack(np64(q), np64(k), hd ** -0.5) <= 0.8 * so.W
    qc, vc = q.cuda(), v.cuda()
    for j in [1] + list(range(168, 176)):  # a sink, and every column modulo 8
        bad = k.clone()
        _key(bad[0], j, kind)
        o, lse = ttcd.sink_window_attn(qc, bad.cuda(), vc, window, n_sink, lse=True)
        _compare(o[0], lse[0], q[0], bad[0], v[0], np.arange(T), window, n_sink, (kind, j))
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("L,window", [(400, 150), (2600, 2500)])
def test_paged(ttcd, kind, hd, L, window):
    """The tiled kernel (one chunk, alone and beside a token) and the one of few rows."""
    Hq, Hkv, page, n = 4, 2, 16, 40
    g = torch.Generator().manual_seed(hd + L)
    k, v = (torch.randn(L, Hkv, hd, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(n, Hq, hd, generator=g).bfloat16()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = lambda x: x.view(-1, page, Hkv, hd).transpose(1, 2).contiguous().cuda()  # noqa: E731
    pad = -L % page
    zeros = torch.zeros(pad, Hkv, hd, dtype=torch.bfloat16)
    vp = pages(torch.cat([v, zeros]))
    table = torch.arange((L + pad) // page, dtype=torch.int32).expand(2, -1).contiguous().cuda()
    qc = q.cuda()
    for j in [1] + list(range(L - 72, L - 64)):
        bad = k.clone()
        _key(bad, j, kind)
        kp = pages(torch.cat([bad, zeros]))
        for new, seqs, max_q in (([n], 1, n), ([n - 1, 1], 2, n - 1), ([n], 1, 1)):
            starts = i32(*np.concatenate([[0], np.cumsum(new)]).tolist())
            o, lse = ttcd.paged_window_attn(qc, kp, vp, table[:seqs].contiguous(), starts,
                                            i32(*[L] * seqs), window, 4, max_q=max_q, lse=True)
            row = 0
            for m in new:
                _compare(o[row:row + m], lse[:, row:row + m], q[row:row + m], bad, v,
                         np.arange(L - m, L), window, 4, (kind, j, new, max_q))
                row += m
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("T", [1, 200])
def test_a_row_of_minus_infinities_is_nan(ttcd, T):
    q = torch.full((1, T, 2, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((1, T, 1, 64), -INF, dtype=torch.bfloat16, device="cuda")
    o, lse = ttcd.sink_window_attn(q, k, q[:, :, :1].contiguous(), 50, 2, lse=True)
    assert torch.isnan(o).all() and (lse == -INF).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window,n_sink", [(300, 0), (60, 4)])
def test_gradients_of_a_query_that_is_nan(ttcd, hd, window, n_sink):
    """Its own dq and the dk and dv of all keys that it sees are NaN, in every column."""
    T = 260
    q, k, v = (x.cuda() for x in make_attention_inputs(1, T, 2, 1, hd, seed=9))
    d_o = torch.randn(1, T, 2, hd, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = ttcd.sink_window_attn(q, k, v, window, n_sink, lse=True)
    clean = ttcd.sink_window_attn_backward(q, k, v, o, lse, d_o, window, n_sink)
    for t in range(200, 204):
        for h in range(2):
            bad = q.clone()
            bad[0, t, h] = NAN
            o, lse = ttcd.sink_window_attn(bad, k, v, window, n_sink, lse=True)
            assert torch.isnan(o[0, t, h]).all() and torch.isnan(lse[0, h, t])
            dq, dk, dv, ws = ttcd.sink_window_attn_backward(bad, k, v, o, lse, d_o, window, n_sink)
            see = torch.from_numpy(so.mask([t], np.arange(T), window, n_sink)[0]).cuda()
            assert torch.isnan(dq[0, t, h]).all()
            assert torch.isnan(dk[0, see]).all() and torch.isnan(dv[0, see]).all()
            # P of a hidden key is 0 and d_o is finite
            assert torch.equal(dv[0, ~see], clean[2][0, ~see])
            # another tile's rows have nothing to do with it
            assert torch.equal(dq[0, :64], clean[0][0, :64])
            assert ttcd.check_device_status(ws) == ttcd.OK
