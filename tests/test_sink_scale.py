"""The backward refuses a softmax scale whose inverse it cannot form (on the host:
nothing is launched, the pointers are never dereferenced)."""
import dual_window_attention_b200 as ttcd
from dual_window_attention_b200 import build

P = 1 << 20


def test_tiny_scale():
    build.build()
    lib = ttcd.load_library()
    sizes = (2, 100, 4, 2, 64, 10, 4)
    for scale in (1e-31, 1e-38, 1e-45):
        assert lib.ttcd_sink_window_attn_backward(*[P] * 9, *sizes, scale, P, 1 << 40,
                                                  None) == ttcd.ERR_UNSUPPORTED
