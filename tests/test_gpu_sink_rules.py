"""Branches of the launch rules that ordinary sizes take: a backward whose first key
tile alone is cut into parts, and the kernel of few rows with one or two tiles in
flight, alone and beside the tiled kernel, with its keys split or not.  The rules are
written out here for the 148 SMs of a B200, so that a case says which branch it takes."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from tests.test_gpu_paged import Batch
from tests.test_gpu_sink_attention import _inputs, _within
from ttcd_workloads import make_attention_inputs

SMS = 148


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    from dual_window_attention_b200 import build
    build.build()
    m.load_library()
    return m


# ------------------------------------------------------------------ backward
BACKWARD = [
    # B, T, Hq, Hkv, hd, window, n_sink, items of far queries
    (1, 1400, 16, 8, 128, 700, 4, 1),     # far items beside a first tile in two parts
    (1, 1400, 16, 8, 64, 2000, 9, 0),     # a window beyond the sequence: none
    (1, 2000, 15, 5, 64, 600, 128, 2),    # groups of 3, a tile of sinks, two items
    (2, 3000, 4, 2, 64, 750, 1, 3),       # three
]


def _plan(B, T, Hq, Hkv, hd, window, n_sink):
    """(parts of the first key tile, of the others, far items) of the backward."""
    cdiv = lambda a, b: -(-a // b)  # noqa: E731
    tpt, n_kt = 128 // (Hq // Hkv), cdiv(T, 128)
    visits = cdiv(min(window + 127, T), tpt)
    parts = max(1, min(SMS // (B * Hkv * n_kt), visits // 6))
    parts0 = 2 * parts if n_sink and visits >= 12 and B * Hkv * n_kt < 2 * SMS else parts
    far = cdiv(T, tpt) - (min(T - 1, window + 126) // tpt + 1) if n_sink else 0
    items = cdiv(far, max(4 if parts > 1 else 16, cdiv(visits, parts0), cdiv(far, 64))) if far > 0 else 0
    return parts0, parts, items


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink,far", BACKWARD)
def test_cases_cut_the_first_key_tile_alone(ttcd, B, T, Hq, Hkv, hd, window, n_sink, far):
    assert _plan(B, T, Hq, Hkv, hd, window, n_sink) == (2, 1, far)
    # and the library's plan is this one: its workspace holds two parts of 128 rows
    row = B * Hkv * 2 * hd * 4
    n_qt = -(-T // (128 // (Hq // Hkv)))
    want = ttcd.STATUS_BYTES + B * Hkv * n_qt * 256 * 16 + 2 * row * 128 + ((1 + far) * n_sink * row if far else 0)
    assert ttcd.load_library().ttcd_sink_window_attn_backward_workspace_size(B, T, Hq, Hkv, hd, window,
                                                                             n_sink) == want


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,hd,window,n_sink,far", BACKWARD)
def test_backward_with_the_first_key_tile_in_parts(ttcd, B, T, Hq, Hkv, hd, window, n_sink, far):
    q, k, v = _inputs(B, T, Hq, Hkv, hd, seed=T)
    d_o = make_attention_inputs(B, T, Hq, 1, hd, seed=13)[0]
    qc, kc, vc, gc = q.cuda(), k.cuda(), v.cuda(), d_o.cuda()
    o, lse = ttcd.sink_window_attn(qc, kc, vc, window, n_sink, lse=True)
    got = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink)
    assert ttcd.check_device_status(got[3]) == ttcd.OK
    g, e = so.sink_window_attention_vjp(np64(q), np64(k), np64(v), np64(d_o), window, n_sink, hd ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        _within(x, g[n], e[n], n)
    again = ttcd.sink_window_attn_backward(qc, kc, vc, o, lse, gc, window, n_sink)
    assert all(torch.equal(x, y) for x, y in zip(got[:3], again[:3]))


# ------------------------------------------------------------------ few rows
def _units(hd, units, keys):
    """(tiles in flight, CTAs per unit) of the kernel of few rows with 8 rows."""
    def splits(held):
        most = min(16, keys // 64 if units <= held else keys // 2048)
        s = 1
        while 2 * s <= most and (2 * s * units <= held if units <= held else s * units < 4 * held):
            s *= 2
        return s
    held1, held2 = ({32: 4, 64: 4, 128: 3}[hd] * SMS, {32: 4, 64: 3, 128: 2}[hd] * SMS)
    s1, s2 = splits(held1), splits(held2)
    one = hd != 32 and units <= held1 and (units > held2 or s1 >= 2 * s2)
    return (1, s1) if one else (2, s2)


FEW = [
    # sequences, Hq, Hkv, hd, keys in the window, page, chunk beside them, (tiles, CTAs)
    (65, 4, 2, 64, 2100, 64, 0, (1, 4)),
    (64, 4, 2, 64, 2100, 16, 150, (1, 4)),      # beside the tiled kernel
    (80, 4, 2, 128, 1500, 64, 0, (1, 2)),
    (79, 4, 2, 128, 1500, 32, 90, (1, 2)),
    (230, 2, 2, 64, 300, 32, 0, (1, 1)),        # more units than two tiles in flight hold
    (230, 4, 2, 128, 4200, 128, 0, (2, 2)),     # more than the GPU holds at once, split
    (310, 4, 2, 64, 4200, 128, 0, (2, 2)),
    (309, 4, 2, 64, 4200, 128, 40, (2, 2)),
    (150, 16, 4, 32, 4200, 64, 0, (2, 2)),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,hd,window,page,chunk,rule", FEW)
def test_cases_take_the_named_variants(seqs, Hq, Hkv, hd, window, page, chunk, rule):
    tokens = 8 // (Hq // Hkv)
    capacity = -(-(window + 400) // page) * page
    assert _units(hd, (seqs + (chunk > 0)) * Hkv, min(window + tokens + 4, capacity)) == rule


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,Hq,Hkv,hd,window,page,chunk,rule", FEW)
def test_few_rows(ttcd, seqs, Hq, Hkv, hd, window, page, chunk, rule):
    """Single tokens of sequences of many lengths that share the pages of one context,
    and a chunk of it where one stands beside them; hidden rows and pages hold NaN only
    behind the context's end."""
    n_sink, g = 4, torch.Generator().manual_seed(seqs + hd)
    L = window + 400
    k, v = (torch.randn(L, Hkv, hd, generator=g).bfloat16() for _ in range(2))
    lens = torch.randint(1, L + 1, (seqs,), generator=g).tolist()
    new = [1] * seqs
    lens[0] = L
    if chunk:
        lens, new = lens + [L], new + [chunk]
    q = torch.randn(sum(new), Hq, hd, generator=g).bfloat16()
    pad = torch.full((-L % page, Hkv, hd), float("nan")).bfloat16()
    kp, vp = (torch.cat([x, pad]).view(-1, page, Hkv, hd).transpose(1, 2).contiguous().cuda() for x in (k, v))
    table = torch.arange(len(kp), dtype=torch.int32).expand(len(lens), -1).contiguous().cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    call = lambda: ttcd.paged_window_attn(q.cuda(), kp, vp, table, i32(starts), i32(lens), window, n_sink,  # noqa: E731
                                          max_q=max(new), lse=True)
    o, lse = call()
    assert ttcd.get_device_error()[0] == ttcd.OK
    for h in range(Hq):
        for rows, t in ((slice(0, seqs), np.array(lens[:seqs]) - 1), (slice(seqs, None), np.arange(L - chunk, L))):
            if len(t) == 0:
                continue
            ro, rl, _, bo = so.attend(np64(q[rows, h]), np64(k[:, h * Hkv // Hq]), np64(v[:, h * Hkv // Hq]), t,
                                      np.arange(L), window, n_sink, hd ** -0.5)
            _within(o[rows, h], ro, bo, ("o", h))
            _within(lse[h, rows], rl, so.W + 2.0 ** -22 * np.abs(rl), ("lse", h))
    o2, lse2 = call()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ------------------------------------------------------------------ both kernels
@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,hd,page", [(6, 2, 64, 16), (4, 2, 128, 64)])
def test_a_mixed_batch_and_its_two_kinds_alone(ttcd, Hq, Hkv, hd, page):
    """The chunks of a mixed batch alone, and its single tokens alone: each within the
    oracle's bound, and so within twice that bound of its rows in the batch."""
    lens, new, window, n_sink = [900, 300, 1000, 77, 640, 1200], [200, 1, 1, 77, 1, 3], 500, 4
    b = Batch(lens, new, Hq, Hkv, hd, page, window, n_sink, seed=3)
    o, lse = b.attend(ttcd, lse=True)
    b.check(o, lse)
    starts = np.concatenate([[0], np.cumsum(new)])
    for kind in ([s for s, n in enumerate(new) if n > 3], [s for s, n in enumerate(new) if n <= 3]):
        rows = torch.cat([torch.arange(starts[s], starts[s + 1]) for s in kind]).cuda()
        part = [new[s] for s in kind]
        qs = torch.tensor(np.concatenate([[0], np.cumsum(part)]), dtype=torch.int32).cuda()
        alone, alone_lse = ttcd.paged_window_attn(b.q.cuda()[rows].contiguous(), b.k_pages, b.v_pages,
                                                  b.table[kind].contiguous(), qs, b.kv_len[kind].contiguous(),
                                                  window, n_sink, max_q=max(part), lse=True)
        row = 0
        for s in kind:
            n, L = new[s], lens[s]
            for h in range(Hq):
                ro, rl, _, bo = so.attend(np64(b.q[starts[s]:starts[s + 1], h]), np64(b.k[s][:, h * Hkv // Hq]),
                                          np64(b.v[s][:, h * Hkv // Hq]), np.arange(L - n, L), np.arange(L),
                                          window, n_sink, hd ** -0.5)
                _within(alone[row:row + n, h], ro, bo, ("alone", s, h))
                _within(alone_lse[h, row:row + n], rl, so.W + 2.0 ** -22 * np.abs(rl), ("lse", s, h))
                _within(alone[row:row + n, h], np64(o[starts[s]:starts[s + 1], h]), 2 * bo, ("batch", s, h))
            row += n
    assert ttcd.get_device_error()[0] == ttcd.OK
