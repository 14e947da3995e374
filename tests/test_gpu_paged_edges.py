"""Calls of the paged cache at the ends of what it takes: positions of half a billion,
batches without any new token, tables that name a page twice, other forms of `lse`."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from tests.test_gpu_paged import Batch
from tests.test_gpu_sink_attention import _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hd,n", [(64, 1), (64, 70), (128, 1), (128, 70), (32, 2)])
def test_far_positions(ttcd, hd, n):
    """Write and attend at positions just below 2^30, where the pages between the sinks
    and the window are long gone."""
    page, window, n_sink, Hq, Hkv, theta = 128, 200, 4, 4, 2, 1e6
    max_pages = (1 << 30) // page - 1
    L = max_pages * page - 3
    g = torch.Generator().manual_seed(hd + n)
    first = (L - n - window) // page
    held = [0, *range(first, max_pages)]
    kp, vp = (torch.randn(len(held) + 1, Hkv, page, hd, generator=g).bfloat16() for _ in range(2))
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    for i, p in enumerate(held):
        table[0, p] = i
    qkv = torch.randn(n, (Hq + 2 * Hkv) * hd, generator=g).bfloat16()
    kc, vc = kp.cuda(), vp.cuda()
    args = (table, _i32(0, n), _i32(L))
    q = ttcd.paged_kv_append(qkv.cuda(), kc, vc, *args, Hq, rope_theta=theta)
    x, pos = np64(qkv).reshape(n, -1, hd), np.arange(L - n, L)
    rot = so.rotate(x[:, :Hq + Hkv], pos, theta)
    # the write's own bound, and the angle in 64 bits: 2^30 radians times a few 2^-53
    half = hd // 2
    big = np.maximum(np.abs(x[:, :Hq + Hkv, :half]), np.abs(x[:, :Hq + Hkv, half:]))
    tol = so.U * np.abs(rot) + (2.0 ** -20 + 2.0 ** -20) * np.concatenate([big, big], -1)
    _within(q, rot[:, :Hq], tol[:, :Hq], "q")
    rows = [(held.index(p // page), p % page) for p in pos]
    for i, (at, r) in enumerate(rows):
        _within(kc[at, :, r], rot[i, Hq:], tol[i, Hq:], "k")
        assert torch.equal(vc[at, :, r].cpu(), qkv[i].view(-1, hd)[Hq + Hkv:])
    j = np.concatenate([np.arange(n_sink), np.arange(L - n - window + 1, L)])
    at, r = torch.tensor([held.index(p // page) for p in j]), torch.tensor(j % page)
    k, v = np64(kc.cpu()[at, :, r]), np64(vc.cpu()[at, :, r])
    for max_q in {1, n}:
        o, lse = ttcd.paged_window_attn(q, kc, vc, *args, window, n_sink, max_q=max_q, lse=True)
        for h in range(Hq):
            ro, rl, _, bo = so.attend(np64(q[:, h]), k[:, h // 2], v[:, h // 2], pos, j, window, n_sink, hd ** -0.5)
            _within(o[:, h], ro, bo, ("o", h, max_q))
            _within(lse[h], rl, so.W + 2.0 ** -22 * np.abs(rl), ("lse", h, max_q))
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("max_q", [1, 100])
def test_no_sequence_has_new_tokens(ttcd, max_q):
    """All rows are padding: nothing is written, and nothing is wrong."""
    kp = torch.full((3, 2, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp, table = kp.clone(), _i32(*[-1] * 8).view(2, 4)
    rows = torch.full((5, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(rows, 7.0), torch.full((4, 5), 7.0, device="cuda")
    ttcd.paged_window_attn(rows, kp, vp, table, _i32(0, 0, 0), _i32(30, 0), 10, 2, max_q=max_q, o=o, lse=lse)
    ttcd.paged_kv_append(rows.new_zeros(5, 8 * 64), kp, vp, table, _i32(0, 0, 0), _i32(30, 0), 4, q=o)
    assert (o == 7).all() and (lse == 7).all() and torch.isnan(kp).all() and torch.isnan(vp).all()
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("max_q", [1, 64])
def test_a_page_that_a_table_names_twice(ttcd, max_q):
    """Its keys count at each of their positions."""
    b = Batch([96], [40], 4, 2, 64, 16, 96, 0, seed=2)
    b.table[0, 1], b.table[0, 3] = b.table[0, 0], b.table[0, 0]
    for x in (b.k[0], b.v[0]):
        x[16:32], x[48:64] = x[:16].clone(), x[:16].clone()
    b.check(*b.attend(ttcd, lse=True, max_q=max_q))
    assert ttcd.get_device_error()[0] == ttcd.OK


def test_lse_is_given_for_any_true_value(ttcd):
    b = Batch([90, 200], [60, 1], 4, 2, 64, 16, 50, 4)
    o, lse = b.attend(ttcd, lse=True)
    for yes in (1, np.True_):
        assert torch.equal(b.attend(ttcd, lse=yes)[1], lse)
    for no in (False, 0, None):
        o2, none = b.attend(ttcd, lse=no)
        assert none is None and torch.equal(o2, o)
