"""The extend step and the attention that reads its workspace: the cached NVFP4 prefix and the chunk written by
nvfp4_kv_extend_step, then nvfp4_paged_extend_attention over the FP8 workspace with the tensors' scales."""
import numpy as np
import pytest
import torch

import plain_steps
import plain_windows
from test_gpu_extend_attention import Chunk
from test_gpu_fp8_pages import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("D,T,G", [(64, 16, 4), (128, 64, 4), (256, 32, 2), (128, 16, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
def test_prefix_and_chunk(kv, cuda, D, T, G, window, sinks):
    H, prefix, chunk = 2, [4, 0, 20, 1], [3 * T + 7, 90, T, 1]
    lens = [a * T + n for a, n in zip(prefix, chunk)]
    c = Chunk(cuda, lens, chunk, H, T, D, G, seed=D + T, blocks=False)
    g = c.g
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    pages = [-(-n // T) for n in chunk]
    cached, fresh = sum(prefix), sum(pages)
    slots = lambda first, n: [int(c.table[b, j]) for b in range(4) for j in range(first[b], first[b] + n[b])]  # noqa: E731
    pool = cached + fresh + 3   # of NVFP4 pages: the prefixes first, then the chunks'
    kd, ks = u(0, 256, pool, H, T, D // 2).to(cuda), u(0x28, 0x39, pool, H, T, D // 16).to(cuda)
    vd, vs = u(0, 256, pool, H, T // 2, D).to(cuda), u(0x28, 0x39, pool, H, T // 2, D // 16, 2).to(cuda)
    gk, gv, wk, wv = (torch.tensor([x], device=cuda) for x in (0.5, 0.25, 0.011, 0.007))
    ws = [torch.zeros((c.P, H, T, D), dtype=torch.uint8, device=cuda) for _ in range(2)]
    new = [torch.randn((fresh, H, T, D), generator=g).to(torch.bfloat16).to(cuda) for _ in range(2)]
    lay = c.layout(kv)
    part = lambda layout, scale, data, sc, w, x, s: dict(  # noqa: E731
        layout=layout, global_scale=scale, data=data, scales=sc, prefix_page_ids=i32(list(range(cached))), ws=w,
        ws_prefix_ids=i32(slots([0] * 4, prefix)), ws_chunk_ids=i32(slots(prefix, pages)), chunk=x,
        chunk_dst_ids=i32(list(range(cached, cached + fresh))), ws_scale=s)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    before = plain_steps.keys(kd.cpu().numpy(), ks.cpu().numpy()) * 0.5, values(vd.cpu().numpy(), vs.cpu().numpy()) * 0.25
    kv.nvfp4_kv_extend_step([part(lay, gk, kd, ks, ws[0], new[0], wk),
                             part(lay.with_packing(kv.PACK_TOKEN_PAIRS), gv, vd, vs, ws[1], new[1], wv)], status=status)
    c.window, c.sinks, c.k, c.v, c.ks, c.vs = window, sinks, ws[0].cpu(), ws[1].cpu(), wk.cpu(), wv.cpu()
    got = c.run(kv, status=status)
    assert status.item() == 0
    c.check(got)
    # what the workspace holds is the cache and the chunk, each to half a step of E4M3 (or of its subnormals) of the tensor's scale
    for x, codes, scale, old in ((new[0], c.k, 0.011, before[0]), (new[1], c.v, 0.007, before[1])):
        want = np.concatenate([old[:cached], x.double().cpu().numpy()])
        have = plain_windows.FP8[codes.numpy()[slots([0] * 4, prefix) + slots(prefix, pages)]] * float(np.float32(scale))
        want = np.clip(want, -448 * scale, 448 * scale)
        assert (np.abs(have - want) <= np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -20)).all()
