"""A step with too few free pages: the sequences that are served come out as if the others were not there, the others keep
their length and pages, have no slots, and are served when pages have come back."""
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


def test_a_step_with_too_few_pages(kv, cuda):
    H, G, D, T, maxp, P = 2, 4, 128, 16, 12, 11
    hq, rows, B = H * G, 200, 4
    g = torch.Generator().manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    lay, status = kv.Layout(H, D, T), i32([0])
    lens, table = i32([0] * B), i32([[-1] * maxp] * B)
    stack, count = torch.randperm(P, generator=g).to(torch.int32).to(cuda), i32([P])
    starts, slots, positions = i32([0] * (B + 1)), torch.zeros(rows, dtype=torch.int64, device=cuda), i32([0] * rows)
    hot = [torch.zeros((P, H, T, D), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    fp8 = [torch.zeros((P, H, T, D), dtype=torch.uint8, device=cuda) for _ in range(2)]
    scales = [torch.ones((P, H), device=cuda) for _ in range(2)]
    sm = float(np.float32(D ** -0.5))

    def step(new, seed):
        r = torch.Generator().manual_seed(seed)
        status.zero_()
        kv.nvfp4_kv_step_tables(lay, lens, i32(new), stack, count, table, lens, starts, slots, positions, status=status)
        n = int(starts[-1])
        q, k, v = (torch.randn((rows, h, D), generator=r).to(torch.bfloat16).to(cuda) for h in (hq, H, H))
        here = slots[:n] >= 0
        page, tok = slots[:n][here] // T, slots[:n][here] % T
        hot[0][page, :, tok], hot[1][page, :, tok] = k[:n][here], v[:n][here]
        ids = torch.where(torch.arange(maxp, device=cuda) * T < lens[:, None], table, -1).flatten().contiguous()
        tokens = (lens[:, None] - torch.arange(maxp, device=cuda) * T).clamp(0, T).int().flatten().contiguous()
        for a, b, s in zip(hot, fp8, scales):
            kv.nvfp4_kv_fp8_pages(lay, a, b, s, src_page_ids=ids, dst_page_ids=ids, page_tokens=tokens, status=status)
        out, lse = torch.zeros((rows, hq, D), dtype=torch.bfloat16, device=cuda), torch.zeros((rows, hq), device=cuda)
        kv.nvfp4_paged_extend_attention(lay, q, *fp8, table, lens, starts, sm, out, k_block_scales=scales[0], v_block_scales=scales[1], lse=lse, status=status)
        c = Cache.__new__(Cache)
        c.fmt, c.T, c.D, c.P, c.lens, c.table = "fp8", T, D, P, lens.tolist(), table.cpu()
        (c.k, c.v), (c.kb, c.vb), c.ks, c.vs = [x.cpu() for x in fp8], [x.cpu() for x in scales], None, None
        for b, a in enumerate(new):   # served rows against 64 bits
            at = int(starts[b])
            if a <= 0 or int(slots[at]) < 0:
                continue
            for h in range(H):
                kk, vv, ok = c.tokens(b, h)
                see = np.repeat(plain_windows.visible(c.lens[b] - a + np.arange(a), c.lens[b], 0, 0), G, 0)
                sl = slice(h * G, (h + 1) * G)
                plain_windows.check((out[at:at + a, sl].double().cpu().numpy().reshape(-1, D), lse[at:at + a, sl].double().cpu().numpy().reshape(-1)),
                                    q[at:at + a, sl].double().cpu().numpy().reshape(-1, D), kk, vv, see, sm, np.abs(vv).max(), blocks=True)
        return int(status), lens.tolist(), slots.cpu(), out, lse

    assert step([40, 70, 3, 16], 1)[:2] == (0, [40, 70, 3, 16]) and count.item() == 1  # 3 + 5 + 1 + 1 of 11 pages
    # 9 more tokens need a page, 60 more need four, one more none, one more one
    s, now, slot, out, lse = step([9, 60, 1, 1], 2)
    assert s == kv.STATUS_NO_PAGES and now == [49, 70, 4, 16] and count.item() == 0
    assert (slot[:9] >= 0).all() and (slot[9:69] == -1).all() and slot[69] >= 0 and slot[70] == -1
    # more rows than it has tokens: not a row of it is made up
    s, now, slot, out, lse = step([1, 1, 1, 100], 3)
    assert s == kv.STATUS_NO_PAGES | kv.STATUS_BAD_SEQ_LEN and now == [50, 71, 5, 16]
    assert (slot[3:103] == -1).all() and not bool(out[3:103].any()) and bool((lse[3:103] == -float("inf")).all())
    # one ends, and its pages serve the others
    s, now, slot, out, lse = step([-1, 9, 1, 1], 4)
    assert s == 0 and now == [0, 80, 6, 17] and (slot[:11] >= 0).all()
