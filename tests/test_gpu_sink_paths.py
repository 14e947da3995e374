"""The sink-window and paged kernels where their launch rules change: keys split
over clusters, single tiles and pairs, one or two kernels for a batch, and what
must not depend on them (bits of a repeated backward, other scales, strides refused)."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from tests.test_gpu_paged import Batch
from tests.test_gpu_sink_attention import _inputs, _within
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", [
    (1, 2900, 1, 1, 64, 2500, 4),     # few pairs of tiles, many keys: clusters
    (1, 2900, 3, 1, 128, 2000, 128),  # the same with groups of 3 and a tile of sinks
    (1, 2100, 2, 1, 32, 1 << 30, 0),  # causal, head_dim 32
    (1, 1250, 16, 8, 128, 700, 9),    # pairs without clusters
    (2, 2000, 10, 5, 64, 700, 9),
])
def test_dense_forward(ttcd, B, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T)
    o, lse = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), window, n_sink, lse=True)
    assert ttcd.get_device_error()[0] == ttcd.OK
    ro, rl, bo = so.sink_window_attention(np64(q), np64(k), np64(v), window, n_sink, hd ** -0.5)
    _within(o, ro, bo, "o")
    _within(lse, rl, so.W + 2.0 ** -22 * np.abs(rl), "lse")


@pytest.mark.parametrize("lens,new,Hq,Hkv,hd,page,window,n_sink", [
    ([4000], [300], 2, 1, 64, 16, 3000, 4),               # one chunk: clusters of the tiled kernel
    ([5000, 4200], [1, 260], 8, 2, 128, 128, 2600, 100),  # beside a single token
    ([3900, 40, 3500, 7], [9, 1, 8, 2], 4, 2, 128, 64, 3000, 4),   # just above and at a unit
    ([2600], [1], 12, 1, 64, 32, 2500, 4),                # groups of 12: units of 16 rows
    ([2600, 900], [2, 1], 12, 1, 128, 32, 2500, 4),       # and two tokens of them: tiled
    ([2600], [1], 24, 1, 128, 16, 2500, 4),               # groups of 24: tiled, clusters
    ([9000] * 3, [1] * 3, 4, 2, 128, 64, 8192, 4),        # wide clusters of the small kernel
])
def test_paged_attention(ttcd, lens, new, Hq, Hkv, hd, page, window, n_sink):
    b = Batch(lens, new, Hq, Hkv, hd, page, window, n_sink, seed=hd)
    for max_q in (max(new), 1, 64):
        b.check(*b.attend(ttcd, lse=True, max_q=max_q))
        assert ttcd.get_device_error()[0] == ttcd.OK


def test_a_mixed_batch_is_its_sequences_alone(ttcd):
    """Chunks and single tokens together: bit for bit what each of the two kernels
    gives for its sequences."""
    lens, new = [900, 300, 1000, 77, 640], [200, 1, 1, 77, 1]
    b = Batch(lens, new, 6, 2, 64, 16, 500, 4, seed=3)
    o, lse = b.attend(ttcd, lse=True)
    b.check(o, lse)
    again, _ = b.attend(ttcd, lse=True)
    assert torch.equal(o, again)
    ones = [i for i, n in enumerate(new) if n == 1]
    at = torch.tensor([sum(new[:i]) for i in ones]).cuda()
    q = b.q.cuda()[at].contiguous()
    qs = torch.arange(len(ones) + 1, dtype=torch.int32).cuda()
    alone, _ = ttcd.paged_window_attn(q, b.k_pages, b.v_pages, b.table[ones].contiguous(), qs,
                                      b.kv_len[ones].contiguous(), 500, 4, max_q=1)
    # another split of the keys rounds the merged sums elsewhere: a bf16 step
    torch.testing.assert_close(alone.float(), o[at].float(), rtol=2.0 ** -7, atol=2.0 ** -9)


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", [
    (1, 2600, 4, 2, 64, 100, 7),     # many items of far queries
    (2, 1100, 6, 2, 128, 64, 128),   # and a tile of sinks, groups of 3
    (1, 900, 2, 2, 64, 1, 1),
])
def test_backward_far_items_and_repeated_bits(ttcd, B, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T)
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=11)[0]
    qc, kc, vc, gc = q.cuda(), k.cuda(), v.cuda(), d_o.cuda()
    o, lse = ttcd.sink_window_attn(qc, kc, vc, window, n_sink, lse=True)
    first = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink)
    g, e = so.sink_window_attention_vjp(np64(q), np64(k), np64(v), np64(d_o), window, n_sink, hd ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), first):
        _within(x, g[n], e[n], n)
    for _ in range(3):
        again = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink,
                                               workspace=first[3])
        assert all(torch.equal(x, y) for x, y in zip(first[:3], again[:3]))
    assert ttcd.check_device_status(first[3]) == ttcd.OK


@pytest.mark.parametrize("scale", [0.01, 0.3])
def test_other_scales(ttcd, scale):
    B, T, Hq, Hkv, hd, window, n_sink = 1, 400, 4, 2, 64, 150, 4
    q, k, v = make_attention_inputs(B, T, Hq, Hkv, hd, seed=21)
    assert so.score_slack(np64(q), np64(k), scale) <= 0.8 * so.W
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=22)[0]
    o, lse = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), window, n_sink, scale=scale, lse=True)
    ro, rl, bo = so.sink_window_attention(np64(q), np64(k), np64(v), window, n_sink, scale)
    _within(o, ro, bo, "o")
    _within(lse, rl, so.W + 2.0 ** -22 * np.abs(rl), "lse")
    got = ttcd.sink_window_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, d_o.cuda(), window,
                                         n_sink, scale=scale)
    g, e = so.sink_window_attention_vjp(np64(q), np64(k), np64(v), np64(d_o), window, n_sink, scale)
    for n, x in zip(("dq", "dk", "dv"), got):
        _within(x, g[n], e[n], n)


def test_backward_leaves_other_rows_alone(ttcd):
    """dk and dv of a sequence that ends inside a tile: nothing behind it is written."""
    q, k, v = (x.cuda() for x in make_attention_inputs(1, 200, 4, 2, 64, seed=5))
    o, lse = ttcd.sink_window_attn(q, k, v, 60, 4, lse=True)
    lib = ttcd.load_library()
    pool = [torch.full((1, 400, h, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    need = lib.ttcd_sink_window_attn_backward_workspace_size(1, 200, 4, 2, 64, 60, 4)
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
    ws[:ttcd.STATUS_BYTES] = 0
    g = torch.ones_like(q)
    status = lib.ttcd_sink_window_attn_backward(
        *[x.data_ptr() for x in (q, k, v, o, lse, g, *pool)], 1, 200, 4, 2, 64, 60, 4, 0.0,
        ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == ttcd.OK and (ws[need:] == 7).all()
    for x in pool:
        assert torch.isfinite(x).all() and (x[:, 200:] == 7).all()


def test_captured_training_step_beside_eager_ones(ttcd):
    """One captured forward and backward, replayed on one stream while eager calls run
    on another: each has its own workspace."""
    q, k, v = (x.cuda() for x in make_attention_inputs(1, 900, 4, 2, 64, seed=6))
    g = torch.randn_like(q)
    def step():
        o, lse = ttcd.sink_window_attn(q, k, v, 120, 4, lse=True)
        return (o, lse) + ttcd.sink_window_attn_backward(q, k, v, o, lse, g, 120, 4)[:3]
    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    other = torch.cuda.Stream()
    for _ in range(5):
        graph.replay()
        with torch.cuda.stream(other):
            eager = step()
        torch.cuda.synchronize()
        for a, b, c in zip(want, out, eager):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink", [
    (1, 1500, 4, 1, 64, 1500, 4),     # few key tiles, many queries each: cut into parts
    (1, 1700, 6, 1, 128, 800, 128),   # and far items of a tile of sinks
    (2, 700, 16, 1, 64, 500, 0),      # 8 tokens a tile, parts that have no visits
])
def test_backward_in_parts(ttcd, B, T, Hq, Hkv, hd, window, n_sink):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T)
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=12)[0]
    qc, kc, vc, gc = q.cuda(), k.cuda(), v.cuda(), d_o.cuda()
    o, lse = ttcd.sink_window_attn(qc, kc, vc, window, n_sink, lse=True)
    got = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink)
    g, e = so.sink_window_attention_vjp(np64(q), np64(k), np64(v), np64(d_o), window, n_sink, hd ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        _within(x, g[n], e[n], n)
    again = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink)
    assert all(torch.equal(x, y) for x, y in zip(got[:3], again[:3]))


@pytest.mark.parametrize("window", [1 << 30, 1 << 31, (1 << 32) + 7, 1 << 62])
def test_a_window_of_any_length_is_causal(ttcd, window):
    q, k, v = (x.cuda() for x in make_attention_inputs(1, 300, 4, 2, 64, seed=8))
    o, lse = ttcd.sink_window_attn(q, k, v, 300, 4, lse=True)
    wide, wide_lse = ttcd.sink_window_attn(q, k, v, window, 4, lse=True)
    assert torch.equal(o, wide) and torch.equal(lse, wide_lse)
    want = ttcd.sink_window_attn_backward(q, k, v, o, lse, q, 300, 4)
    got = ttcd.sink_window_attn_backward(q, k, v, o, lse, q, window, 4)
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("Hq", [2, 12])
def test_a_sink_with_most_of_the_weight_is_not_rounded_twice(ttcd, hd, Hq):
    """Key 0 has almost all of every row's weight p_0.  With weights that are off by
    r_j, |r_j| <= U, and the sum of the same weights below, the result is off by at most
    2 U (1 - p_0) |v_0| + 2 U sum_{j > 0} p_j |v_j| (over 1 - U), beside its own rounding
    U |o| and the 32-bit work W: the rounding of p_0 must not show."""
    T, window, page = 304, 40, 16
    g = torch.Generator().manual_seed(hd)
    q, k, v = (torch.randn(1, T, h, hd, generator=g) for h in (Hq, 1, 1))
    q *= 0.5
    q[..., 0] += 6
    k[:, 0] = 0
    k[:, 0, :, 0] = 10 * hd ** 0.5 / 6
    q, k, v = (x.bfloat16() for x in (q, k, v))
    # the exponential adds 2.8e-6 and 2^-22 of a score (below 24): 0.07 W
    assert so.score_slack(np64(q), np64(k), hd ** -0.5) <= 0.9 * so.W
    t, vs = np.arange(T), np.abs(np64(v)[0, :, 0])
    refs, bounds = [], []
    for h in range(Hq):
        ro, _, p, _ = so.attend(np64(q)[0, :, h], np64(k)[0, :, 0], np64(v)[0, :, 0], t, t, window, 1,
                                hd ** -0.5)
        assert np.median(p[:, 0]) > 0.99
        refs.append(ro)
        others = (1 - p[:, :1]) * vs[:1] + p[:, 1:] @ vs[1:]
        bounds.append(so.U * np.abs(ro) + 2 * so.U / (1 - so.U) * others + so.W * (p @ vs))
    ref, bound = np.stack(refs, 1), np.stack(bounds, 1)
    o, _ = ttcd.sink_window_attn(q.cuda(), k.cuda(), v.cuda(), window, 1)
    _within(o[0], ref, bound, "dense")
    # single tokens at every position, over pages that all sequences share
    k_pages, v_pages = (x[0].view(T // page, page, 1, hd).transpose(1, 2).contiguous().cuda() for x in (k, v))
    table = torch.arange(T // page, dtype=torch.int32).expand(T, -1).contiguous().cuda()
    one, _ = ttcd.paged_window_attn(q[0].cuda(), k_pages, v_pages, table,
                                    torch.arange(T + 1, dtype=torch.int32).cuda(),
                                    torch.arange(1, T + 1, dtype=torch.int32).cuda(), window, 1, max_q=1)
    _within(one, ref, bound, "paged")
    # and one chunk of them all
    chunk, _ = ttcd.paged_window_attn(q[0].cuda(), k_pages, v_pages, table[:1].contiguous(),
                                      torch.tensor([0, T], dtype=torch.int32).cuda(),
                                      torch.tensor([T], dtype=torch.int32).cuda(), window, 1, max_q=T)
    _within(chunk, ref, bound, "chunk")


def test_more_sequences_than_one_search_step(ttcd):
    """1100 sequences of none to three new tokens: the write gives the bits that calls of
    20 sequences give, and the attention is the oracle's through either kernel."""
    g = torch.Generator().manual_seed(31)
    new = torch.randint(0, 4, (1100,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(1, 30, (1100,), generator=g))]
    b = Batch(lens, new, 2, 1, 64, 16, 12, 2, seed=4)
    for max_q in (1, 64):
        b.check(*b.attend(ttcd, lse=True, max_q=max_q))
    table = torch.arange(b.table.numel(), dtype=torch.int32).view(b.table.shape).cuda()
    qkv = torch.randn(b.total, 4 * 64, generator=g).bfloat16().cuda()
    pools = [torch.zeros(table.numel(), 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    q = ttcd.paged_kv_append(qkv, *pools[:2], table, b.q_start, b.kv_len, 2)
    for s in range(0, 1100, 20):
        at = b.q_start[s:s + 21]
        lo, hi = at[0].item(), at[-1].item()
        part = ttcd.paged_kv_append(qkv[lo:hi], *pools[2:], table[s:s + 20], (at - lo).contiguous(),
                                    b.kv_len[s:s + 20].clone(), 2)
        assert torch.equal(part, q[lo:hi])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert pools[0].any() and ttcd.get_device_error()[0] == ttcd.OK
