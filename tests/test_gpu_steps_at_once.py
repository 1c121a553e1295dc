"""Decode steps of two caches at once: every call of a step (append, page bounds, selection, attention) runs beside the
other cache's calls on another stream, and has the results of a step alone."""
import pytest
import torch

from test_gpu_sparse import Steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def test_steps_of_two_caches_on_two_streams(kv, cuda):
    both = [Steps(kv, cuda, seed=3), Steps(kv, cuda, seed=4, H=1, G=5, D=128, T=32, maxp=9, budget=5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(60):
        fed = []
        for s, stream in zip(both, streams):
            with torch.cuda.stream(stream):
                fed.append(s.feed([i, i, i]))
        for s, stream in zip(both, streams):
            with torch.cuda.stream(stream):
                s.launch()
        torch.cuda.synchronize()
        for s, x in zip(both, fed):
            s.plain(x)


def test_two_selections_at_once(kv, cuda):
    """One long sequence on each stream: clusters of 8 CTAs of both calls beside one another."""
    D, T, H, G, budget, maxp, P = 128, 16, 2, 4, 200, 6000, 900
    g = torch.Generator(device=cuda).manual_seed(5)
    bounds = torch.randint(-60, 60, (P, H, 2, D), generator=g, device=cuda, dtype=torch.int8)
    bounds = torch.stack([bounds.amax(2), bounds.amin(2)], 2).contiguous()
    scales = torch.rand((P, H), generator=g, device=cuda) + 0.5
    lay, lens = kv.Layout(H, D, T), torch.tensor([maxp * T - 5], dtype=torch.int32, device=cuda)
    tables = [torch.randint(0, P, (1, maxp), generator=g, device=cuda, dtype=torch.int32) for _ in range(2)]
    qs = [torch.randn((1, H * G, D), generator=g, device=cuda).to(torch.bfloat16) for _ in range(2)]

    def outs():
        return [torch.full((1, H, budget), 7, dtype=torch.int32, device=cuda) for _ in range(2)] + [
            torch.full((1, H), 7, dtype=torch.int32, device=cuda)]

    def call(i, o, stream=None):
        kv.nvfp4_kv_select_pages(lay, qs[i], bounds, scales, tables[i], lens, o[0], o[2], sink_pages=2, recent_pages=3,
                                 sel_index=o[1], stream=stream)
    want = [outs(), outs()]
    for i in range(2):
        call(i, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [outs(), outs()]
        torch.cuda.synchronize()
        for i in range(2):
            call(i, got[i], streams[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
