"""Calls that take their scratch from the allocator themselves, on streams other than the current one, while the
current stream and others allocate and write blocks of the same size: the results are those of a call alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


class Attention:
    """160 pairs of up to 4096 tokens: cut into runs over all pairs, whose records go through the workspace."""

    def __init__(self, kv, dev, dense):
        B, H, G, D, T, pages = 20, 8, 1, 64, 64, 64
        g = torch.Generator(device=dev).manual_seed(1)
        u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
        n = 200
        one = torch.ones(1, device=dev)
        self.kv, self.dense, self.lay = kv, dense, kv.Layout(H, D, T)
        self.q = torch.randn((B, H * G, D), generator=g, device=dev).to(torch.bfloat16)
        self.pool = (u(0, 256, n, H, T, D // 2), u(0x28, 0x39, n, H, T, D // 16), one,
                     u(0, 256, n, H, T // 2, D), u(0x28, 0x39, n, H, T // 2, D // 16, 2), one)
        lead = (B,) if dense else (B, H)
        self.table = torch.randint(0, n, (*lead, pages), generator=g, device=dev, dtype=torch.int32)
        self.lens = torch.randint(pages * T // 2, pages * T + 1, lead, generator=g, device=dev, dtype=torch.int32)
        self.bytes = (kv.nvfp4_paged_decode_workspace_size(self.lay, B, H * G, pages) if dense else
                      kv.nvfp4_paged_sparse_decode_workspace_size(self.lay, B, H * G, pages))

    def result(self):
        return torch.zeros_like(self.q)

    def call(self, out, **kw):
        f = self.kv.nvfp4_paged_decode_attention if self.dense else self.kv.nvfp4_paged_sparse_decode_attention
        f(self.lay, self.q, *self.pool, self.table, self.lens, 0.125, out, **kw)


class GlobalScale:
    def __init__(self, kv, dev):
        self.kv, self.lay = kv, kv.Layout(8, 128, 64)
        self.src = torch.randn((64, 8, 64, 128), device=dev).to(torch.bfloat16)
        self.bytes = kv.nvfp4_kv_global_scale_workspace_size()

    def result(self):
        return torch.zeros(1, device=self.src.device)

    def call(self, out, **kw):
        self.kv.nvfp4_kv_compute_global_scale(self.lay, self.src, out, **kw)


def make(kind, kv, dev):
    return GlobalScale(kv, dev) if kind == "global scale" else Attention(kv, dev, kind == "dense")


def alone(c, dev):
    """The result over a workspace of the caller; it has to have been written (else the case shows nothing)."""
    w = torch.full((c.bytes,), 0xA5, dtype=torch.uint8, device=dev)
    want = c.result()
    c.call(want, workspace=w)
    torch.cuda.synchronize()
    assert bool((w != 0xA5).any())
    return want


@pytest.mark.parametrize("handles", [False, True])
@pytest.mark.parametrize("kind", ["selected pages", "dense", "global scale"])
def test_own_scratch_on_two_side_streams(kv, cuda, kind, handles):
    c = make(kind, kv, cuda)
    want = alone(c, cuda)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [c.result() for _ in range(20)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        s = streams[i % 2]
        c.call(out, stream=s.cuda_stream if handles else s)
        junk = [torch.full((max(c.bytes, 16),), 0xFF, dtype=torch.uint8, device=cuda) for _ in range(3)]
        del junk
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["selected pages", "dense", "global scale"])
def test_own_scratch_taken_behind_work_of_the_current_stream(kv, cuda, kind):
    """Blocks that the current stream still writes when the host has let go of them are not the side stream's."""
    c = make(kind, kv, cuda)
    want = alone(c, cuda)
    side = torch.cuda.Stream()
    outs = [c.result() for _ in range(10)]
    torch.cuda.synchronize()
    for out in outs:
        busy = torch.zeros(64 << 20, dtype=torch.float32, device=cuda)
        for _ in range(4):
            busy.add_(1)
        late = torch.full((max(c.bytes, 16),), 0xFF, dtype=torch.uint8, device=cuda)
        del late, busy
        c.call(out, stream=side)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["selected pages", "dense", "global scale"])
def test_own_scratch_captured_on_a_side_stream(kv, cuda, kind):
    """A graph captured on a side stream keeps its scratch (it lies in the graph's memory)."""
    c = make(kind, kv, cuda)
    want, out, side = alone(c, cuda), c.result(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call(out, stream=side)
    for _ in range(3):
        out.zero_()
        junk = torch.full((max(c.bytes, 16),), 0xFF, dtype=torch.uint8, device=cuda)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk
