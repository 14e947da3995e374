"""Refusals of the sink-window and paged entry points, on the host: nothing is
launched for them, so they need no GPU (the pointers are never dereferenced)."""
import pytest
import torch

import dual_window_attention_b200 as ttcd

P = 1 << 20  # aligned, never dereferenced
OK_DENSE = dict(B=2, T=100, Hq=4, Hkv=2, hd=64, window=10, n_sink=4, scale=0.0, dtype=ttcd.BF16)
OK_PAGED = dict(n_seq=3, total_q=20, max_q=9, n_pages=50, page_size=16, max_pages=8, Hq=4, Hkv=2,
                hd=64, window=10, n_sink=4, scale=0.0, dtype=ttcd.BF16)
INVALID, UNSUPPORTED = ttcd.ERR_INVALID_ARG, ttcd.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from dual_window_attention_b200 import build
    build.build()
    return ttcd.load_library()


SHAPE_REFUSALS = [
    (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(window=0), INVALID),
    (dict(n_sink=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(dtype=7), INVALID), (dict(dtype=ttcd.F32), UNSUPPORTED),
    (dict(hd=48), UNSUPPORTED), (dict(hd=256), UNSUPPORTED), (dict(n_sink=129), UNSUPPORTED),
    (dict(Hq=258, Hkv=2), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", SHAPE_REFUSALS + [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(B=1 << 12, T=1 << 20), UNSUPPORTED)])
def test_dense_forward(lib, change, status):
    a = {**OK_DENSE, **change}
    assert lib.ttcd_sink_window_attn(P, P, P, P, None, *[a[n] for n in OK_DENSE], None) == status


@pytest.mark.parametrize("at", range(5))
def test_dense_forward_pointers(lib, at):
    for bad in ([None, P + 8] if at < 4 else [P + 8]):
        p = [P] * 5
        p[at] = bad
        assert lib.ttcd_sink_window_attn(*p, *OK_DENSE.values(), None) == INVALID


@pytest.mark.parametrize("change,status", [
    (c, s) for c, s in SHAPE_REFUSALS if "dtype" not in c] + [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(hd=32), UNSUPPORTED),
    (dict(B=1 << 12, T=1 << 20), UNSUPPORTED)])
def test_dense_backward(lib, change, status):
    a = {**OK_DENSE, **change}
    sizes = [a[n] for n in ("B", "T", "Hq", "Hkv", "hd", "window", "n_sink")]
    assert lib.ttcd_sink_window_attn_backward(*[P] * 9, *sizes, a["scale"], P, 1 << 40,
                                              None) == status
    if "scale" not in change:
        assert lib.ttcd_sink_window_attn_backward_workspace_size(*sizes) == 0


def test_dense_backward_pointers_and_workspace(lib):
    sizes = [OK_DENSE[n] for n in ("B", "T", "Hq", "Hkv", "hd", "window", "n_sink")]
    need = lib.ttcd_sink_window_attn_backward_workspace_size(*sizes)
    assert need >= ttcd.STATUS_BYTES
    f = lib.ttcd_sink_window_attn_backward
    for at in range(9):
        for bad in (None, P + 8):
            p = [P] * 9
            p[at] = bad
            assert f(*p, *sizes, 0.0, P, need, None) == INVALID
    assert f(*[P] * 9, *sizes, 0.0, None, need, None) == INVALID
    assert f(*[P] * 9, *sizes, 0.0, P, need - 1, None) == ttcd.ERR_WORKSPACE


PAGED_REFUSALS = [
    (dict(n_seq=0), INVALID), (dict(total_q=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(n_pages=1 << 27), UNSUPPORTED), (dict(max_pages=1 << 26), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", SHAPE_REFUSALS + PAGED_REFUSALS + [(dict(max_q=0), INVALID)])
def test_paged_attention(lib, change, status):
    a = {**OK_PAGED, **change}
    assert lib.ttcd_paged_window_attn(*[P] * 8, *[a[n] for n in OK_PAGED], None) == status


@pytest.mark.parametrize("at", range(8))
def test_paged_attention_pointers(lib, at):
    int32 = 3 <= at <= 5
    for bad in ([None] if at != 7 else []) + [P + (2 if int32 else 4)]:
        p = [P] * 8
        p[at] = bad
        assert lib.ttcd_paged_window_attn(*p, *OK_PAGED.values(), None) == INVALID


APPEND = ("n_seq", "total_q", "n_pages", "page_size", "max_pages", "Hq", "Hkv", "hd")


@pytest.mark.parametrize("change,status", PAGED_REFUSALS + [
    (c, s) for c, s in SHAPE_REFUSALS if not {"window", "n_sink", "scale"} & set(c)] + [
    (dict(theta=-1.0), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(theta=float("inf")), INVALID)])
def test_append(lib, change, status):
    a = {**OK_PAGED, "theta": 1e4, **change}
    assert lib.ttcd_paged_kv_append(*[P] * 7, *[a[n] for n in APPEND], a["theta"], a["dtype"],
                                    None) == status


@pytest.mark.parametrize("at", range(7))
def test_append_pointers(lib, at):
    for bad in (None, P + (2 if at >= 4 else 4)):
        p = [P] * 7
        p[at] = bad
        assert lib.ttcd_paged_kv_append(*p, *[OK_PAGED[n] for n in APPEND], 1e4, ttcd.BF16,
                                        None) == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    q, kv = torch.zeros(1, 9, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ttcd.sink_window_attn(q, kv, kv, 4, 1)
    with pytest.raises(ValueError):
        ttcd.sink_window_attn(q[0], kv, kv, 4, 1)
    with pytest.raises(ValueError):
        ttcd.sink_window_attn_backward(q, kv, kv, q, torch.zeros(1, 4, 9), q, 4, 1)
    pages, i = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ttcd.paged_window_attn(q[0], pages, pages, i[None], torch.zeros(2, dtype=torch.int32), i, 4, 1, 9)
    with pytest.raises(ValueError):
        ttcd.paged_kv_append(torch.zeros(9, 8 * 64, dtype=torch.bfloat16), pages, pages, i[None],
                             torch.zeros(2, dtype=torch.int32), i, 4)


WIDE = [1 << 31, (1 << 32) + 1, -(1 << 32) + 1]


@pytest.mark.parametrize("x", WIDE)
def test_binding_does_not_cut_numbers_to_32_bits(lib, x):
    q, kv = torch.zeros(1, 9, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16)
    pages, i = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    paged = (q[0], pages, pages, i[None], torch.zeros(2, dtype=torch.int32), i)
    lse = torch.zeros(1, 4, 9)
    windows = [x] if x < 0 else []  # a long window is one that hides nothing
    for w, s in [(4, x)] + [(w, 1) for w in windows]:
        name = "n_sink" if s == x else "window"
        with pytest.raises(ValueError, match=name):
            ttcd.sink_window_attn(q, kv, kv, w, s)
        with pytest.raises(ValueError, match=name):
            ttcd.sink_window_attn_backward(q, kv, kv, q, lse, q, w, s)
        with pytest.raises(ValueError, match=name):
            ttcd.paged_window_attn(*paged, w, s, 9)
    with pytest.raises(ValueError, match="max_q"):
        ttcd.paged_window_attn(*paged, 4, 1, x)


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 5
    with pytest.raises(ValueError, match="cuda:1"):
        ttcd._launching(0, Stream())
