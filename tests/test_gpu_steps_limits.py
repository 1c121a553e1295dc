"""Decode-step calls at the ends of what they allow: the most pairs, very long pages, the same token twice, a single
page of everything."""
import numpy as np
import pytest
import torch

import plain_steps
from test_gpu_append import Case, table_of
from test_gpu_attention_numerics import Pool
from test_gpu_sparse import check_selection, some_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def test_attention_over_the_most_pairs(kv, cuda):
    """65535 pairs of 0 to 32 tokens; every 37th one compared, all finite."""
    B, H, T, D = 13107, 5, 16, 64
    c = Pool(cuda, 30, H, T, D, 1).to_device()
    lens = torch.randint(0, 2 * T + 1, (B, H), generator=c.g, dtype=torch.int32)
    table = torch.randint(0, 30, (B, H, 2), generator=c.g, dtype=torch.int32)
    q = torch.randn((B, H, D), generator=c.g).to(torch.bfloat16)
    out, lse = c.sparse(kv, q, table, lens)
    assert np.isfinite(out).all() and np.array_equal(np.isfinite(lse), lens.numpy() > 0)
    some = slice(0, B, 37)
    c.check((out[some], lse[some]), q[some], table[some], lens[some])


def test_selection_over_the_most_pairs(kv, cuda):
    B, H, T, D = 13107, 5, 16, 64
    bounds, scales, g = some_pages(40, H, D, 2)
    table = torch.randint(0, 40, (B, 6), generator=g, dtype=torch.int32)
    lens = torch.randint(0, 6 * T + 1, (B,), generator=g, dtype=torch.int32)
    q = torch.randn((B, H, D), generator=g).to(torch.bfloat16)
    sel = torch.full((B, H, 3), 99, dtype=torch.int32, device=cuda)
    sl = torch.full((B, H), 99, dtype=torch.int32, device=cuda)
    kv.nvfp4_kv_select_pages(kv.Layout(H, D, T), q.to(cuda), bounds.to(cuda), scales.to(cuda), table.to(cuda), lens.to(cuda),
                             sel, sl, sink_pages=1, recent_pages=1)
    some = slice(0, B, 23)
    want = plain_steps.select(q[some].double().numpy(), bounds.numpy(), scales.double().numpy(), table[some].numpy(),
                              lens[some].numpy(), T, 3, 1, 1)
    assert np.array_equal(sel[some].cpu().numpy(), want[1]) and np.array_equal(sl[some].cpu().numpy(), want[2])
    assert bool((sel != 99).all()) and bool((sl != 99).all())


@pytest.mark.parametrize("D,G", [(256, 8), (128, 1)])
def test_selection_at_the_page_limit_of_wide_heads(kv, cuda, D, G):
    bounds, scales, g = some_pages(70, 1, D, D)
    table = torch.randint(0, 70, (1, 49152), generator=g, dtype=torch.int32)
    q = torch.randn((1, G, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor([49152 * 16], dtype=torch.int32), 1, 16, 3000, 1, 1)


def test_selection_of_very_long_pages(kv, cuda):
    """Pages of 2^29 tokens: lengths and selected lengths up to 1.5 2^30."""
    T, D, H = 1 << 29, 64, 2
    bounds, scales, g = some_pages(9, H, D, 3)
    table = torch.randint(0, 9, (4, 3), generator=g, dtype=torch.int32)
    q = torch.randn((4, 2 * H, D), generator=g).to(torch.bfloat16)
    lens = torch.tensor([3 * T, 2 * T + 1, T, 5], dtype=torch.int64).to(torch.int32)
    for budget in (1, 2, 3):
        check_selection(kv, cuda, q, bounds, scales, table, lens, H, T, budget, 0, 1)


def test_append_to_very_long_pages(kv, cuda):
    """Two pages of 2^20 tokens: slots at both ends of each."""
    T, H, D = 1 << 20, 1, 64
    slots = np.array([0, 1, T - 2, T - 1, T, T + 7, 2 * T - 1, 2 * T - 2])
    c = Case(cuda, len(slots), 2, H, D, 2, 1, slots, seed=1)
    pool = [torch.zeros(s, dtype=torch.uint8, device=cuda)
            for s in ((2, H, T, D // 2), (2, H, T, D // 16), (2, H, T // 2, D), (2, H, T // 2, D // 16, 2))]
    kv.nvfp4_kv_append(kv.Layout(H, D, T), c.k, c.v, c.slots.to(cuda), *pool)
    # the same rows in a cache of two-token pages, page by page
    small = {n: np.zeros(s, np.uint8) for n, s in (("kd", (5, H, 2, D // 2)), ("ks", (5, H, 2, D // 16)), ("vd", (5, H, 1, D)),
                                                   ("vs", (5, H, 1, D // 16, 2)))}
    pairs = np.unique(slots // 2)
    where = {int(p): i for i, p in enumerate(pairs)}
    plain_steps.append(small, c.hk, c.hv, [2 * where[int(s) // 2] + int(s) % 2 for s in slots], 2, 1.0, 1.0)
    for p, i in where.items():
        page, t = 2 * p // T, 2 * p % T
        got = [pool[0][page, :, t:t + 2], pool[1][page, :, t:t + 2], pool[2][page, :, t // 2:t // 2 + 1],
               pool[3][page, :, t // 2:t // 2 + 1]]
        for n, x in zip(("kd", "ks", "vd", "vs"), got):
            assert np.array_equal(x.cpu().numpy(), small[n][i]), (n, p)
    assert int(pool[0].count_nonzero()) == int(np.count_nonzero(small["kd"]))
    assert int(pool[2].count_nonzero()) == int(np.count_nonzero(small["vd"]))


@pytest.mark.parametrize("slots", [
    [4, 5, 4, 9, 9, 8], [5, 4, 5, 5, 20, 21], [4, 5, 5, 4, 4, 5, 30], [7, 7, 7, 7, 6, 40], [4, 4, 5, 12, 13, 12, 13]])
def test_the_same_token_twice_touches_no_other(kv, cuda, slots):
    """Rows of one slot: that token is unspecified, every other keeps its value or gets its own row's (among them the
    other token of the V byte); rotated queries do not depend on slots."""
    T, P, H, D = 16, 4, 3, 64
    rot = ("halves", 0, 64, table_of(5000, 64))
    for seed in range(5):
        c = Case(cuda, len(slots), 4, H, D, T, P, slots, seed=seed)
        pool, outs = c.run(kv, rot)
        once = [n for n, s in enumerate(slots) if slots.count(s) == 1]
        want, rows = c.want(rot)
        twice = sorted({s for s in slots if slots.count(s) > 1})
        # only the nibbles and scales of the tokens of `twice` are not compared
        for s in twice:
            page, t = s // T, s % T
            for x in (pool, want):
                x["kd"][page, :, t] = x["ks"][page, :, t] = 0
                x["vs"][page, :, t // 2, :, t % 2] = 0
                x["vd"][page, :, t // 2] &= 0xF0 if t % 2 == 0 else 0x0F
        for n in want:
            assert np.array_equal(pool[n], want[n]), n
        for n in range(len(slots)):
            assert torch.equal(outs[0][n], torch.from_numpy(rows[0][n]).float().to(torch.bfloat16))
        for n in once:
            assert torch.equal(outs[1][n], torch.from_numpy(rows[1][n]).float().to(torch.bfloat16))
            assert torch.equal(outs[2][n], torch.from_numpy(rows[2][n]).float().to(torch.bfloat16))
