"""The scratch that a call without a workspace takes: on which stream it is allocated, seen on the host through
stand-ins for the library, the tensors and the streams (the GPU side is in test_gpu_workspaces.py)."""
import contextlib

import pytest
import torch

import nvfp4_paged_kv_gb300 as kv


class Fake:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, shape, dtype, device=torch.device("cuda", 0)):
        self.shape, self.dtype, self.device = shape, dtype, device

    def get_device(self):
        return 0

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device, self.device_index = handle, torch.device("cuda", 0), 0


@pytest.fixture
def world(monkeypatch):
    """Records the streams that scratch was allocated on and calls were launched on. The current one is 77."""
    w = {"now": [77], "taken": [], "launched": []}

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *a: 4096
            return lambda *a: w["launched"].append(a[-1]) or 0

    @contextlib.contextmanager
    def current(s):
        w["now"].append(s.cuda_stream)
        yield
        w["now"].pop()

    def empty(n, dtype, device):
        w["taken"].append(w["now"][-1])
        return Fake((n,), dtype, device)

    monkeypatch.setattr(kv, "_lib", Lib())
    monkeypatch.setattr(kv, "_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda dev: w["now"][-1])
    monkeypatch.setattr(kv, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(kv, "_dtype_code", lambda t, e: 0)

    @contextlib.contextmanager
    def on_device(tensors, stream):
        yield 77 if stream is None else stream.cuda_stream if isinstance(stream, Stream) else int(stream)

    monkeypatch.setattr(kv, "_on_device", on_device)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", current)
    return w


def calls():
    lay = kv.Layout(2, 64, 16)
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    q, out, g = Fake((3, 4, 64), torch.bfloat16), Fake((3, 4, 64), torch.bfloat16), Fake((1,), f32)
    kd, ks = Fake((5, 2, 16, 32), u8), Fake((5, 2, 16, 4), u8)
    return {
        "selected pages": lambda s: kv.nvfp4_paged_sparse_decode_attention(
            lay, q, kd, ks, g, kd, ks, g, Fake((3, 2, 4), i32), Fake((3, 2), i32), 0.125, out, stream=s),
        "dense": lambda s: kv.nvfp4_paged_decode_attention(
            lay, q, kd, ks, g, kd, ks, g, Fake((3, 4), i32), Fake((3,), i32), 0.125, out, stream=s),
        "global scale": lambda s: kv.nvfp4_kv_compute_global_scale(
            lay, Fake((5, 2, 16, 64), torch.bfloat16), g, stream=s),
    }


@pytest.mark.parametrize("call", list(calls()))
@pytest.mark.parametrize("stream,handle", [(None, 77), (77, 77), (0x5000, 0x5000), ("object", 0x6000), (0, 0), (1, 0)])
def test_scratch_is_allocated_on_the_launch_stream(world, call, stream, handle):
    """A block of the allocator is reused in the order of the stream it was allocated on: on any other than the
    launch stream, its next owner could write it while the call still runs."""
    given = Stream(handle) if stream == "object" else stream
    calls()[call](given)
    assert world["taken"] == [handle]
    assert world["launched"] == [stream if isinstance(stream, int) else handle]


@pytest.mark.parametrize("call", list(calls()))
def test_no_scratch_on_the_per_thread_stream(world, call):
    """Handle 2 is another stream for every thread; no block of the allocator belongs to it."""
    with pytest.raises(ValueError, match="workspace"):
        calls()[call](2)
    assert world["launched"] == []
