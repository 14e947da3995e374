"""Softmax scales and rotary bases that 32 bits cannot hold are refused, on the host:
one that becomes 0 there would silently mean the default scale, or no rotation."""
import pytest
import torch

import dual_window_attention_b200 as ttcd
from dual_window_attention_b200 import build

P = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ttcd.load_library()


@pytest.mark.parametrize("scale", [1e-46, -1e-46, 1e-300])
def test_binding_refuses_what_becomes_zero(lib, scale):
    q, kv = torch.zeros(1, 9, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16)
    pages, i = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    paged = (pages, pages, i[None], torch.zeros(2, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="scale"):
        ttcd.sink_window_attn(q, kv, kv, 4, 1, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        ttcd.sink_window_attn_backward(q, kv, kv, q, torch.zeros(1, 4, 9), q, 4, 1, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        ttcd.paged_window_attn(q[0], *paged, 4, 1, 9, scale=scale)
    with pytest.raises(ValueError, match="rope_theta"):
        ttcd.paged_kv_append(torch.zeros(9, 8 * 64, dtype=torch.bfloat16), *paged, 4, rope_theta=scale)


def test_library_refuses_a_scale_that_overflows_in_base_2(lib):
    dense = (2, 100, 4, 2, 64, 10, 4)
    paged = (3, 20, 9, 50, 16, 8, 4, 2, 64, 10, 4)
    for scale in (2.4e38, 3.4e38):
        assert lib.ttcd_sink_window_attn(P, P, P, P, None, *dense, scale, ttcd.BF16, None) == ttcd.ERR_INVALID_ARG
        assert lib.ttcd_sink_window_attn_backward(*[P] * 9, *dense, scale, P, 1 << 40, None) == ttcd.ERR_INVALID_ARG
        assert lib.ttcd_paged_window_attn(*[P] * 8, *paged, scale, ttcd.BF16, None) == ttcd.ERR_INVALID_ARG
