"""The sink-window and paged calls run on the stream they are given, in whichever
form: an object of torch, one of another library, or a handle (0: the default one)."""
import contextlib

import pytest
import torch

import dual_window_attention_b200 as ttcd


class Foreign:
    """A stream object of another library."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("wrap", [int, Foreign])
def test_handles_become_the_streams_they_name(monkeypatch, wrap):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: ("default", dev))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device.index))
    monkeypatch.setattr(torch.cuda, "stream", contextlib.nullcontext)
    for handle, stream in ((0, ("default", 3)), (1, ("external", 1, 3)), (4096, ("external", 4096, 3))):
        with ttcd._launching(3, wrap(handle)) as s:
            assert s == stream


@pytest.mark.gpu
@pytest.mark.parametrize("wrap", [int, Foreign])
def test_handle_zero_is_the_default_stream(wrap):
    """A call with the default stream's handle comes after that stream's work and before
    what follows there: its inputs are written just before it and overwritten just after."""
    from ttcd_workloads import make_attention_inputs
    q, k, v = (x.cuda() for x in make_attention_inputs(1, 300, 4, 2, 64, seed=1))
    k2, big = torch.flip(k, (1,)), torch.randn(8192, 8192, device="cuda")
    want = ttcd.sink_window_attn(q, k, v, 60, 4)[0]
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    with torch.cuda.stream(default):
        for _ in range(3):
            work = k2.clone()
            for _ in range(4):
                big @ big  # milliseconds
            work.copy_(k)
            got = ttcd.sink_window_attn(q, work, v, 60, 4, stream=wrap(default.cuda_stream))[0]
            work.copy_(k2)
            assert torch.equal(got, want)
    with ttcd._launching(0, wrap(0)):
        assert torch.cuda.current_stream() == default
