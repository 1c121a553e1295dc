"""The calls of a step together, as a serving loop makes them: tables and slots from request lengths, rows appended to the
NVFP4 cache and to 16-bit pages, those encoded as FP8, attention of chunks and of single tokens, requests that end and others
that take their pages."""
import numpy as np
import pytest
import torch

import plain_windows
from test_gpu_window_decode import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("D,T,window,sinks", [(128, 64, 0, 0), (64, 16, 70, 3), (256, 32, 150, 20)])
def test_serving_loop(kv, cuda, D, T, window, sinks):
    """Chunks and decode rows over a shared pool, six steps. The extend attention of every step is checked against 64 bits over
    the FP8 pages as they are, the FP8 pages against their definition over the 16-bit ones, and the window decode of single rows
    over the NVFP4 pages that the append wrote."""
    H, G, B, maxp, P = 2, 4, 4, 12, 30
    hq, rows = H * G, 300
    g = torch.Generator().manual_seed(D)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=cuda)  # noqa: E731
    lay = kv.Layout(H, D, T)
    lens, new, table = i32(B), i32(B), i32(B, maxp) - 1
    stack, count = torch.randperm(P, generator=g).to(torch.int32).to(cuda), torch.tensor([P], dtype=torch.int32, device=cuda)
    starts, slots, positions, full = i32(B + 1), torch.zeros(rows, dtype=torch.int64, device=cuda), i32(rows), i32(B + rows // T)
    status = i32(1)
    # the cache: NVFP4 pools, hot 16-bit pages, and the same as FP8 with a scale for each page and head
    kd, ks, vd, vs = u8(P, H, T, D // 2), u8(P, H, T, D // 16), u8(P, H, T // 2, D), u8(P, H, T // 2, D // 16, 2)
    hot = [torch.zeros((P, H, T, D), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    k8, v8 = u8(P, H, T, D), u8(P, H, T, D)
    kb, vb = torch.ones((P, H), device=cuda), torch.ones((P, H), device=cuda)
    gk, gv = torch.tensor([0.01], device=cuda), torch.tensor([0.01], device=cuda)
    sm = float(np.float32(D ** -0.5))
    plan = [[100, 1, 0, 37], [1, 60, 130, 1], [1, 1, 1, -1], [33, -1, 1, 80], [1, 5, 1, 1], [-1, 1, 1, 1]]
    host_len = [0] * B
    for step in plan:
        step = [a if host_len[b] + max(a, 0) <= maxp * T else 0 for b, a in enumerate(step)]
        new.copy_(torch.tensor(step, dtype=torch.int32))
        before = lens.clone()
        kv.nvfp4_kv_step_tables(lay, lens, new, stack, count, table, lens, starts, slots, positions, full_pages=full, status=status)
        host_len = [0 if a == -1 else n + a for n, a in zip(host_len, step)]
        assert lens.tolist() == host_len
        n = int(starts[-1])
        qkv = torch.randn((rows, (hq + 2 * H) * D), generator=g).to(torch.bfloat16).to(cuda)
        q, k, v = (x.view(rows, -1, D) for x in qkv.split([hq * D, H * D, H * D], 1))
        kv.nvfp4_kv_append(lay, k, v, slots, kd, ks, vd, vs, k_global_scale=gk, v_global_scale=gv, status=status)
        # the same rows into the hot pages, and the pages that they touch into FP8, each with its valid tokens
        at = slots[:n]
        page, tok = at // T, at % T
        hot[0][page, :, tok], hot[1][page, :, tok] = k[:n], v[:n]
        index = torch.arange(maxp, device=cuda)
        valid = (lens[:, None] - index * T).clamp(0, T).int()
        touched = ((index + 1) * T > before[:, None]) & (valid > 0) & (new[:, None] > 0)
        ids = torch.where(touched, table, -1).flatten().contiguous()
        tokens = valid.flatten().contiguous()
        for src, dst, scales in ((hot[0], k8, kb), (hot[1], v8, vb)):
            kv.nvfp4_kv_fp8_pages(lay, src, dst, scales, src_page_ids=ids, dst_page_ids=ids, page_tokens=tokens, status=status)
        for e in torch.nonzero(ids >= 0)[::5, 0].tolist():
            code, s = plain_windows.fp8_page(hot[0][ids[e]].double().cpu().numpy(), int(tokens[e]))
            assert np.array_equal(k8[ids[e]].cpu().numpy(), code) and np.array_equal(kb[ids[e]].double().cpu().numpy(), s)
        out, lse = torch.full((rows, hq, D), float("nan"), dtype=torch.bfloat16, device=cuda), torch.zeros((rows, hq), device=cuda)
        kv.nvfp4_paged_extend_attention(lay, q, k8, v8, table, lens, starts, sm, out, k_block_scales=kb, v_block_scales=vb, window=window,
                                        sink_tokens=sinks, lse=lse, status=status)
        # a decode row of each sequence over the NVFP4 pages
        dout, dlse = torch.zeros((B, hq, D), dtype=torch.bfloat16, device=cuda), torch.zeros((B, hq), device=cuda)
        dq = torch.randn((B, hq, D), generator=g).to(torch.bfloat16).to(cuda)
        kv.nvfp4_paged_window_decode_attention(lay, dq, kd, ks, gk, vd, vs, gv, table, lens, sm, dout, window=window or 10 ** 6,
                                               sink_tokens=sinks, lse=dlse, status=status)
        assert status.item() == 0
        assert bool(torch.isnan(out[n:]).all())
        c = Cache.__new__(Cache)
        c.dev, c.H, c.T, c.D, c.G, c.P, c.maxp, c.sm = cuda, H, T, D, G, P, maxp, sm
        c.table, c.lens, c.window, c.sinks = table.cpu(), host_len, window, sinks
        c.fmt, c.k, c.v, c.kb, c.vb, c.ks, c.vs = "fp8", k8.cpu(), v8.cpu(), kb.cpu(), vb.cpu(), None, None
        first = starts.tolist()
        for b in range(B):
            m = first[b + 1] - first[b]
            for h in range(H if m else 0):
                kk, vv, ok = c.tokens(b, h)
                assert ok.all()
                here = np.repeat(plain_windows.visible(np.arange(host_len[b] - m, host_len[b]), host_len[b], window, sinks), G, 0)
                r, heads = slice(first[b], first[b + 1]), slice(h * G, (h + 1) * G)
                plain_windows.check((out[r, heads].double().cpu().numpy().reshape(-1, D), lse[r, heads].double().cpu().numpy().reshape(-1)),
                                    q[r, heads].double().cpu().numpy().reshape(-1, D), kk, vv, here, sm, c.vmax(), blocks=True)
        c.fmt, c.kd, c.ksc, c.vd, c.vsc, c.gk, c.gv = "nvfp4", kd.cpu(), ks.cpu(), vd.cpu(), vs.cpu(), gk.cpu(), gv.cpu()
        c.q, c.window = dq.cpu(), window or 10 ** 6
        c.check((dout.double().cpu().numpy(), dlse.double().cpu().numpy()))


def test_a_step_as_one_graph(kv, cuda):
    """Tables, FP8 encoding and extend attention captured together and replayed over three steps whose lengths only the GPU
    knows; equal to the same calls made one by one."""
    H, G, D, T, B, maxp, rows = 2, 2, 128, 16, 3, 20, 64
    g = torch.Generator().manual_seed(1)
    lay = kv.Layout(H, D, T)

    def state():
        r = torch.Generator().manual_seed(2)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)  # noqa: E731
        s = dict(lens=i32(B), new=i32(B), table=i32(B, maxp) - 1, stack=(torch.randperm(79, generator=r) + 1).to(torch.int32).to(cuda),
                 count=torch.tensor([79], dtype=torch.int32, device=cuda), starts=i32(B + 1), positions=i32(rows),
                 slots=torch.zeros(rows, dtype=torch.int64, device=cuda), ids=i32(B * maxp), tokens=i32(B * maxp),
                 hot=torch.zeros((80, H, T, D), dtype=torch.bfloat16, device=cuda), k8=torch.zeros((80, H, T, D), dtype=torch.uint8, device=cuda),
                 kb=torch.ones((80, H), device=cuda), q=torch.zeros((rows, H * G, D), dtype=torch.bfloat16, device=cuda),
                 out=torch.zeros((rows, H * G, D), dtype=torch.bfloat16, device=cuda), index=torch.arange(maxp, device=cuda))
        s["ws"] = torch.empty(kv.nvfp4_paged_extend_attention_workspace_size(lay, B, H * G), dtype=torch.uint8, device=cuda)
        return s

    def step(s):
        kv.nvfp4_kv_step_tables(lay, s["lens"], s["new"], s["stack"], s["count"], s["table"], s["lens"], s["starts"], s["slots"], s["positions"])
        at = s["slots"].clamp(min=0)
        keep = (s["slots"] >= 0)[:, None, None]
        old = s["hot"][at // T, :, at % T]
        # (a padding row writes slot 0 back; no live token has it, as page 0 is not handed out)
        s["hot"].index_put_((at // T, torch.zeros_like(at), at % T), torch.where(keep[:, 0], s["q"][:, 0], old[:, 0]))
        valid = (s["lens"][:, None] - s["index"] * T).clamp(0, T).int()
        s["ids"].copy_(torch.where(valid > 0, s["table"], -1).flatten())
        s["tokens"].copy_(valid.flatten())
        kv.nvfp4_kv_fp8_pages(lay, s["hot"], s["k8"], s["kb"], src_page_ids=s["ids"], dst_page_ids=s["ids"], page_tokens=s["tokens"])
        kv.nvfp4_paged_extend_attention(lay, s["q"], s["k8"], s["k8"], s["table"], s["lens"], s["starts"], 0.1, s["out"], k_block_scales=s["kb"],
                                        v_block_scales=s["kb"], workspace=s["ws"])
    a, b = state(), state()
    step(b)   # (warm up: kernels' attributes, the allocator; no sequence has tokens yet)
    b = state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    b2 = state()
    for name, t in b2.items():
        b[name].copy_(t) if name != "ws" else None
    for new in ([20, 1, 0], [1, 30, 7], [-1, 1, 1]):
        q = torch.randn((rows, H * G, D), generator=g).to(torch.bfloat16)
        for s in (a, b):
            s["new"].copy_(torch.tensor(new, dtype=torch.int32))
            s["q"].copy_(q)
        step(a)
        b["ws"].random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        n = int(a["starts"][-1])
        for name in ("lens", "table", "stack", "count", "starts", "slots", "k8", "kb"):
            assert torch.equal(a[name], b[name]), name
        assert torch.equal(a["out"][:n], b["out"][:n]) and bool(torch.isfinite(a["out"][:n]).all())
