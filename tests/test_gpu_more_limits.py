"""The step tables, FP8 pages and attentions at the ends of what they allow: pools past 4 GB, the most sequences, very long
pages, one workspace for calls in turn."""
import numpy as np
import pytest
import torch

import plain_windows
from test_gpu_extend_attention import Chunk
from test_gpu_window_decode import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def test_pages_past_4_gigabytes(kv, cuda):
    """Pages at the top of pools of 5 GB: encoded there, read by the decodes and by the extend attention."""
    H, T, D, G = 8, 64, 128, 4
    P = 5 * 2 ** 30 // (H * T * D)
    c = Chunk(cuda, [500, 130], [100, 1], H, T, D, G, seed=3)
    d = Cache(cuda, "nvfp4", [500, 130], H, T, D, G, window=300, sinks=5, seed=4, drop=False)
    shift = P - c.P
    big = [torch.zeros((P, H, T, D), dtype=torch.uint8, device=cuda) for _ in range(2)]
    scales = [torch.ones((P, H), device=cuda) for _ in range(2)]
    # encoded into the top of the pool from small 16-bit pages
    x = torch.randn((c.P, H, T, D), generator=c.g).to(torch.bfloat16)
    ids = torch.arange(c.P, dtype=torch.int32, device=cuda)
    for pool, sc, src in ((big[0], scales[0], x), (big[1], scales[1], x.flip(0))):
        kv.nvfp4_kv_fp8_pages(c.layout(kv), src.to(cuda), pool, sc, src_page_ids=ids, dst_page_ids=ids + shift)
    c.k, c.v = (p[shift:].cpu() for p in big)
    c.kb, c.vb = (s[shift:].cpu() for s in scales)
    c.ks = c.vs = None
    for e in range(0, c.P, 5):
        code, s = plain_windows.fp8_page(x[e].double().numpy(), T)
        assert np.array_equal(c.k[e].numpy(), code) and np.array_equal(c.kb[e].double().numpy(), s)
    assert not bool(big[0][:shift].any())
    table = torch.where((c.table >= 0) & (c.table < c.P), c.table + shift, c.table).to(cuda)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=cuda)
    out, lse = torch.full_like(c.q_dev, float("nan")), torch.zeros(c.q_dev.shape[:2], device=cuda)
    kv.nvfp4_paged_extend_attention(c.layout(kv), c.q_dev, *big, table, lens, torch.tensor(c.starts, dtype=torch.int32, device=cuda), c.sm, out,
                                    k_block_scales=scales[0], v_block_scales=scales[1], lse=lse)
    c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))
    q = torch.randn((2, H * G, D), generator=c.g).to(torch.bfloat16)
    out, lse = torch.zeros(q.shape, dtype=torch.bfloat16, device=cuda), torch.zeros(q.shape[:2], device=cuda)
    kv.nvfp4_paged_fp8_decode_attention(c.layout(kv), q.to(cuda), *big, table, lens, c.sm, out, k_block_scales=scales[0],
                                        v_block_scales=scales[1], lse=lse)
    c.q = q
    Cache.check(c, (out.double().cpu().numpy(), lse.double().cpu().numpy()))
    # the NVFP4 window decode, codes past 2.5 GB in the same bytes
    pool = [b.view(2 * P, -1)[:, :H * T * D // 2] for b in big]
    kd, vd = (p.reshape(2 * P, H, T, D // 2) for p in pool)
    ks, vs = (torch.zeros((2 * P, H, T, D // 16), dtype=torch.uint8, device=cuda) for _ in range(2))
    top = 2 * P - d.P
    for pool, part in ((kd, d.kd), (ks, d.ksc), (vd, d.vd), (vs, d.vsc)):
        pool[top:] = part.reshape(d.P, *pool.shape[1:]).to(cuda)
    table = torch.where((d.table >= 0) & (d.table < d.P), d.table + top, d.table).to(cuda)
    out, lse = torch.zeros(d.q.shape, dtype=torch.bfloat16, device=cuda), torch.zeros(d.q.shape[:2], device=cuda)
    kv.nvfp4_paged_window_decode_attention(d.layout(kv), d.q.to(cuda), kd, ks, d.gk.to(cuda), vd, vs, d.gv.to(cuda), table, lens, d.sm, out,
                                           window=300, sink_tokens=5, lse=lse)
    d.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


@pytest.mark.parametrize("D", [64, 256])
def test_extend_over_the_most_sequences(kv, cuda, D):
    """65535 sequences of 0 to 40 tokens with 0 to 2 rows each; every 97th compared, all finite."""
    B, T, P, G = 65535, 16, 50, 2
    g = torch.Generator().manual_seed(D)
    lens = torch.randint(0, 41, (B,), generator=g)
    new = torch.minimum(torch.randint(0, 3, (B,), generator=g), lens)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    rows = int(starts[-1])
    c = Cache(cuda, "fp8", [40], 1, T, D, G, seed=1)
    k, v = (torch.randint(0, 0x7F, (P, 1, T, D), generator=g, dtype=torch.uint8) for _ in range(2))
    table = torch.randint(0, P, (B, 3), generator=g, dtype=torch.int32)
    q = torch.randn((rows, G, D), generator=g).to(torch.bfloat16)
    out, lse = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=cuda), torch.zeros(q.shape[:2], device=cuda)
    scale = torch.tensor([0.01], device=cuda)
    kv.nvfp4_paged_extend_attention(kv.Layout(1, D, T), q.to(cuda), k.to(cuda), v.to(cuda), table.to(cuda), lens.int().to(cuda),
                                    starts.int().to(cuda), c.sm, out, k_scale=scale, v_scale=scale, lse=lse)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    f = float(scale.double())
    for b in range(0, B, 97):
        n, m = int(lens[b]), int(new[b])
        if m == 0:
            continue
        ids = table[b, :-(-n // T)].numpy()
        kk, vv = (plain_windows.FP8[x.numpy()[ids, 0]].reshape(-1, D)[:n] * f for x in (k, v))
        r = slice(int(starts[b]), int(starts[b + 1]))
        here = np.repeat(plain_windows.visible(np.arange(n - m, n), n, 0, 0), G, 0)
        plain_windows.check((out[r].reshape(-1, D), lse[r].reshape(-1)), q[r].double().numpy().reshape(-1, D), kk, vv, here, c.sm, 448 * f,
                            blocks=True)


def test_very_long_pages(kv, cuda):
    """One page of 4096 tokens for each sequence."""
    c = Chunk(cuda, [4000, 4096, 1], [30, 1, 1], 2, 4096, 128, 4, seed=2)
    c.check(c.run(kv), some=20)
    d = Cache(cuda, "fp8", [4000, 4096, 1], 2, 4096, 64, 4, window=1000, sinks=70, seed=2)
    d.check(d.run(kv))


def test_one_workspace_for_calls_in_turn(kv, cuda):
    """Extend, FP8 decode and window decode on one stream with one workspace, each leaving it as it is; two captured graphs
    replayed in turn over it."""
    c = Chunk(cuda, [3000, 70], [5, 70], 2, 64, 128, 4, seed=1)
    a = Cache(cuda, "fp8", [3000, 70], 2, 64, 128, 4, seed=2)
    b = Cache(cuda, "nvfp4", [3000, 70], 2, 64, 128, 4, window=2500, sinks=9, seed=3)
    want = [x.run(kv) for x in (c, a, b)]
    ws = torch.randint(0, 256, (64 << 20,), dtype=torch.uint8, device=cuda)
    for _ in range(3):
        for x, w in zip((c, a, b), want):
            got = x.run(kv, workspace=ws)
            assert np.array_equal(w[0], got[0], equal_nan=True) and np.array_equal(w[1], got[1], equal_nan=True)
    i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=cuda)  # noqa: E731
    graphs, outs = [], []
    for x in (a, c):
        pools, scales = x.fp8()
        q = x.q.to(cuda)
        out = torch.zeros(q.shape, dtype=torch.bfloat16, device=cuda)
        args = [x.layout(kv), q, *pools, x.table.to(cuda), i(x.lens)] + ([i(c.starts)] if x is c else []) + [x.sm, out]
        f = kv.nvfp4_paged_extend_attention if x is c else kv.nvfp4_paged_fp8_decode_attention
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(*args, workspace=ws, **scales)
        graphs.append((graph, args, scales)), outs.append(out)
    for _ in range(4):
        for (graph, _, _), out, w in zip(graphs, outs, (want[1], want[0])):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(out.double().cpu().numpy(), w[0])


def test_step_tables_of_one_page_of_one_token(kv, cuda):
    """Pages of one token and of 2^30: slots of any page size."""
    for T in (1, 2 ** 30):
        B = 3
        i = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
        past, new, table = [0, 1, 0], [1, 1 if T > 1 else 0, -1], [[-1], [7], [-1]]
        t = dict(stack=i([4, 5, 6]), count=i([3]), table=i(table), lens=i([9] * B), starts=i([9] * (B + 1)), positions=i([9] * 3),
                 slots=torch.full((3,), 9, dtype=torch.int64, device=cuda), left=i([9]), full=i([9] * 6))
        kv.nvfp4_kv_step_tables(kv.Layout(1, 64, T), i(past), i(new), t["stack"], t["count"], t["table"], t["lens"], t["starts"], t["slots"],
                                t["positions"], free_left=t["left"], full_pages=t["full"])
        want = plain_windows.step_tables(past, new, [4, 5, 6], 3, table, T, 3, 6)
        for name in ("lens", "starts", "slots", "positions", "full", "table", "stack"):
            assert t[name].tolist() == want[name], (T, name)


def test_extend_of_many_shapes_on_two_streams(kv, cuda):
    """Drawn shapes, each four times on two streams with scratch of their own: the same result, nothing flagged, nothing NaN."""
    import random
    r = random.Random(7)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(300):
        D, H, G, T = r.choice((64, 128, 256)), r.randint(1, 8), r.randint(1, 8), r.choice((16, 32, 48, 64, 128))
        lens = [r.randint(0, int(2 ** r.uniform(0, 11))) for _ in range(r.choice((1, 2, 5, 17, 40)))]
        new = [r.choice((0, 1, min(n, r.randint(0, 600)))) if n else 0 for n in lens]
        pages = [-(-n // T) for n in lens]
        P = sum(pages) + 1
        if P * H * T * D > 10 ** 8:
            continue
        k, v = (torch.randn((P, H, T, D), device=cuda).to(torch.float8_e4m3fn) for _ in range(2))
        table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32)
        ids, at = torch.randperm(P).int(), 0
        for b, m in enumerate(pages):
            table[b, :m] = ids[at:at + m]
            at += m
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
        starts = i32([sum(new[:b]) for b in range(len(new) + 1)])
        q = torch.randn((max(1, sum(new)), H * G, D), device=cuda).to(torch.bfloat16)
        args = kv.Layout(H, D, T), q, k, v, table.to(cuda), i32(lens), starts, D ** -0.5
        more = dict(window=r.choice((0, 0, 1, 100, 1000)), sink_tokens=r.choice((0, 4, 200)), status=status)
        outs = [torch.zeros_like(q) for _ in range(4)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            kv.nvfp4_paged_extend_attention(*args, o, stream=streams[i % 2], **more)
        torch.cuda.synchronize()
        assert status.item() == 0 and bool(torch.isfinite(outs[0]).all())
        assert all(torch.equal(o, outs[0]) for o in outs[1:])
