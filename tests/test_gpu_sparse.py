"""GPU page bounds, page selection and attention over selected pages against their plain 64-bit forms.

Bounds, scales, scores and selections are exact (their FP32 roundings are part of the definitions, the
sums are integers). Attention has the dense decode's tolerance on BF16 outputs: max-abs 1e-2 on top of
the output's own rounding (half a BF16 step of the exact value), mean-abs 1e-3, LSE within 1e-3: the
probabilities are rounded to FP16 (2^-11 relative each) before the product with values of magnitude up
to a few units, and the other roundings are FP32."""
import numpy as np
import pytest
import torch

import plain_steps

pytestmark = pytest.mark.gpu

MAX_ABS, MEAN_ABS, LSE_ABS = 1e-2, 1e-3, 1e-3


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def rand_u8(shape, g, lo=0, hi=256):
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8)


def k_pool(P, H, T, D, seed, lo=0x18, hi=0x45):
    g = torch.Generator().manual_seed(seed)
    return rand_u8((P, H, T, D // 2), g), rand_u8((P, H, T, D // 16), g, lo, hi)


# ------------------------------------------------------------------------------------ bounds

def check_bounds(kv, cuda, kd, ks, ids, tokens, expect=0):
    P, H, T, D = kd.shape[0], kd.shape[1], kd.shape[2], kd.shape[3] * 2
    bounds = torch.full((P, H, 2, D), 77, dtype=torch.int8, device=cuda)
    scales = torch.full((P, H), -5.0, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    as32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    kv.nvfp4_kv_page_bounds(kv.Layout(H, D, T), kd.to(cuda), ks.to(cuda), bounds, scales, page_ids=as32(ids),
                            page_tokens=as32(tokens), status=status)
    bounds, scales = bounds.cpu().numpy(), scales.cpu().numpy()
    want_b, want_s = np.full_like(bounds, 77), np.full_like(scales, -5.0)
    ids = list(range(P)) if ids is None else ids
    for i, page in enumerate(ids):
        n = T if tokens is None else tokens[i]
        if 0 <= page < P and 0 <= n <= T:
            want_b[page, :, 0], want_b[page, :, 1], want_s[page] = plain_steps.page_bounds(
                kd[page].numpy(), ks[page].numpy(), n)
    assert np.array_equal(scales, want_s)
    assert np.array_equal(bounds, want_b)
    assert status.item() == expect


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H", [(16, 3), (48, 2), (64, 8), (80, 2), (128, 1), (272, 1)])
def test_bounds_of_full_and_partial_pages(kv, cuda, D, T, H):
    kd, ks = k_pool(11, H, T, D, T * D)
    check_bounds(kv, cuda, kd, ks, None, None)
    check_bounds(kv, cuda, kd, ks, [4, 9, 0, 7, 2], [T, 0, 1, (T + 1) // 2, max(0, T - 1)])


def test_bounds_of_every_scale(kv, cuda):
    """Block scales over the whole E4M3 range, zero and subnormal among them; tokens past the page's end
    hold NaN scales."""
    P, H, T, D = 40, 2, 16, 128
    kd, ks = k_pool(P, H, T, D, 1, 0, 0x7F)
    ks[3] = 0
    ks[5] = 1
    kd[7] = 0x88   # minus zero
    ks[:, :, 12:] = 0x7F
    check_bounds(kv, cuda, kd, ks, list(range(P)), [12] * P)


def test_bounds_padding_and_bad_pages(kv, cuda):
    kd, ks = k_pool(6, 2, 16, 64, 2)
    check_bounds(kv, cuda, kd, ks, [-1, 2, -1, 2, 5], None)
    check_bounds(kv, cuda, kd, ks, [6, 1, -7], None, kv.STATUS_PAGE_OOB)
    check_bounds(kv, cuda, kd, ks, [0, 1, 3], [17, -1, 4], kv.STATUS_BAD_SEQ_LEN)


def test_bounds_of_many_pages(kv, cuda):
    """More (page, head) items than one wave of warps, through shuffled ids."""
    P, H, T, D = 9000, 8, 16, 64
    kd, ks = k_pool(P, H, T, D, 3)
    bounds = torch.zeros((P, H, 2, D), dtype=torch.int8, device=cuda)
    scales = torch.zeros((P, H), device=cuda)
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(cuda)
    kv.nvfp4_kv_page_bounds(kv.Layout(H, D, T), kd.to(cuda), ks.to(cuda), bounds, scales, page_ids=ids)
    v = plain_steps.keys(kd.numpy(), ks.numpy())
    top, low = v.max(2), v.min(2)
    s = plain_steps.f32(np.maximum(np.abs(top), np.abs(low)).max(-1) / 127)
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), s)
    d = np.where(s > 0, s, 1)[..., None]
    assert np.array_equal(bounds[:, :, 0].cpu().numpy(), np.minimum(127, np.ceil(plain_steps.f32(top / d))).astype(np.int8))
    assert np.array_equal(bounds[:, :, 1].cpu().numpy(), np.maximum(-127, np.floor(plain_steps.f32(low / d))).astype(np.int8))


# ------------------------------------------------------------------------------------ selection

def selection(kv, cuda, q, bounds, scales, table, lens, H, T, budget, sink, recent, status=None, stream=None):
    B, Hq, D = q.shape
    sel = torch.full((B, H, budget), 99, dtype=torch.int32, device=cuda)
    index = torch.full_like(sel, 99)
    sl = torch.full((B, H), 99, dtype=torch.int32, device=cuda)
    scores = torch.full((B, H, table.shape[1]), 3.5, device=cuda)
    kv.nvfp4_kv_select_pages(kv.Layout(H, D, T), q.to(cuda), bounds.to(cuda), scales.to(cuda), table.to(cuda),
                             lens.to(cuda), sel, sl, sink_pages=sink, recent_pages=recent, sel_index=index,
                             scores=scores, status=status, stream=stream)
    torch.cuda.synchronize()
    return index.cpu().numpy(), sel.cpu().numpy(), sl.cpu().numpy(), scores.cpu().numpy()


def check_selection(kv, cuda, q, bounds, scales, table, lens, H, T, budget, sink, recent, expect=0):
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = selection(kv, cuda, q, bounds, scales, table, lens, H, T, budget, sink, recent, status)
    want = plain_steps.select(q.double().numpy(), bounds.numpy(), scales.double().numpy(), table.numpy(), lens.numpy(), T,
                              budget, sink, recent)
    assert np.array_equal(got[3], np.where(np.isnan(want[3]), 3.5, want[3]).astype(np.float32))
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[2], want[2])
    assert status.item() == expect
    # without the optional outputs: the same selection
    B = q.shape[0]
    sel = torch.full((B, H, budget), 99, dtype=torch.int32, device=cuda)
    sl = torch.full((B, H), 99, dtype=torch.int32, device=cuda)
    kv.nvfp4_kv_select_pages(kv.Layout(H, q.shape[2], T), q.to(cuda), bounds.to(cuda), scales.to(cuda), table.to(cuda),
                             lens.to(cuda), sel, sl, sink_pages=sink, recent_pages=recent)
    assert np.array_equal(sel.cpu().numpy(), want[1]) and np.array_equal(sl.cpu().numpy(), want[2])


def some_pages(P, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    mid, wide = torch.randn((P, H, 1, D), generator=g) * 15, torch.rand((P, H, 1, D), generator=g) * 60
    bounds = torch.cat([mid + wide, mid - wide], 2).round().clamp(-127, 127).to(torch.int8)
    return bounds, torch.rand((P, H), generator=g) * 0.05 + 0.01, g


@pytest.mark.parametrize("D,H,G", [(64, 2, 1), (128, 3, 8), (256, 1, 5), (128, 1, 4)])
@pytest.mark.parametrize("T,budget,sink,recent", [(16, 9, 1, 2), (64, 1, 0, 1), (48, 33, 3, 1), (1, 40, 0, 7)])
def test_selection_of_ragged_sequences(kv, cuda, D, H, G, T, budget, sink, recent):
    """Empty, one-token, shorter than the budget, just longer, long; a partial last page."""
    lens = [0, 1, T * budget, T * budget + 1, T * 200, T * 150 + 1, max(1, T // 2)]
    B, maxp = len(lens), 201
    bounds, scales, g = some_pages(B * 30, H, D, D + T)
    table = torch.randint(0, B * 30, (B, maxp), generator=g, dtype=torch.int32)
    q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor(lens, dtype=torch.int32), H, T, budget, sink, recent)


@pytest.mark.parametrize("B,H,maxp", [(1, 1, 40000), (1, 8, 3000), (3, 30, 700), (40, 8, 130), (1, 2, 129)])
def test_selection_over_clusters_of_every_size(kv, cuda, B, H, maxp):
    """One pair of 40,000 pages to 320 pairs: clusters of 8, 4, 2 and 1 CTAs."""
    D, T, G = 64, 16, 2
    bounds, scales, g = some_pages(1000, H, D, maxp)
    table = torch.randint(0, 1000, (B, maxp), generator=g, dtype=torch.int32)
    lens = torch.randint(maxp * T // 2, maxp * T + 1, (B,), generator=g, dtype=torch.int32)
    q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, lens, H, T, 64, 1, 2)


def test_selection_at_the_page_limit(kv, cuda):
    """49,152 table entries; every page of the pool appears many times, so whole runs of pages tie and
    the lowest win."""
    D, T, H, maxp = 64, 16, 1, 49152
    bounds, scales, g = some_pages(50, H, D, 5)
    table = torch.randint(0, 50, (1, maxp), generator=g, dtype=torch.int32)
    q = torch.randn((1, 1, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor([maxp * T - 3], dtype=torch.int32), H, T, 1000, 2, 3)


def test_ties_go_to_the_lowest_page(kv, cuda):
    D, T, H = 128, 32, 2
    bounds, scales, g = some_pages(3, H, D, 7)
    table = torch.tensor([[0, 1, 2] * 100], dtype=torch.int32)
    q = torch.randn((1, 4, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor([300 * T], dtype=torch.int32), H, T, 77, 0, 1)
    check_selection(kv, cuda, q * 0, bounds, scales, table, torch.tensor([300 * T], dtype=torch.int32), H, T, 20, 1, 1)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_are_exact_at_their_largest(kv, cuda, D):
    """Every product at 255 * 127 with the same sign, then off by one in single dims: sums up to 2^23
    that differ in their last bit are told apart."""
    P, T = 64, 16
    bounds = torch.full((P, 1, 2, D), 127, dtype=torch.int8)
    for i in range(P):
        bounds[i, 0, :, i % D] = 127 - i // 2
    bounds[1::2] *= -1
    scales = torch.full((P, 1), 1.0)
    table = torch.arange(P, dtype=torch.int32)[None]
    for q in (torch.full((1, 2, D), 255.0), torch.full((1, 2, D), -255.0)):
        q[0, 1, ::3] = 1
        check_selection(kv, cuda, q.to(torch.bfloat16), bounds, scales, table, torch.tensor([P * T], dtype=torch.int32), 1, T, 13, 0, 1)


def test_selection_with_queries_that_are_not_finite(kv, cuda):
    """A head with an infinity or a NaN scores 0 everywhere (its group's other heads still decide)."""
    D, T, H, G = 64, 16, 1, 3
    bounds, scales, g = some_pages(60, H, D, 8)
    table = torch.arange(60, dtype=torch.int32)[None].repeat(3, 1)
    q = torch.randn((3, G, D), generator=g)
    q[0, 1, 5], q[1, 0, 0], q[1, 2, 63] = float("inf"), float("nan"), float("-inf")
    q[2] = float("nan")
    check_selection(kv, cuda, q.to(torch.bfloat16), bounds, scales, table, torch.tensor([900, 960, 955], dtype=torch.int32), H, T, 10, 1, 1)


def test_selection_bad_lengths_and_page_ids(kv, cuda):
    D, T, H = 64, 16, 2
    bounds, scales, g = some_pages(50, H, D, 9)
    table = torch.randint(0, 50, (3, 40), generator=g, dtype=torch.int32)
    q = torch.randn((3, 4, D), generator=g).to(torch.bfloat16)
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor([-1, 640, 641], dtype=torch.int32), H, T, 6, 1, 1,
                    kv.STATUS_BAD_SEQ_LEN)
    table[1, 7], table[1, 20], table[2, 3] = 50, -1, 2 ** 31 - 1
    check_selection(kv, cuda, q, bounds, scales, table, torch.tensor([600, 640, 640], dtype=torch.int32), H, T, 38, 1, 1,
                    kv.STATUS_PAGE_OOB)


@pytest.mark.parametrize("B,H,maxp", [(1, 1, 2000), (2, 3, 600), (9, 8, 300)])
def test_selection_captured_and_replayed(kv, cuda, B, H, maxp):
    """Clusters of several CTAs in a CUDA graph on a side stream; lengths and queries change between
    replays, down to sequences that fit the budget."""
    D, T, G, budget = 128, 16, 4, 24
    bounds, scales, g = some_pages(400, H, D, maxp)
    table = torch.randint(0, 400, (B, maxp), generator=g, dtype=torch.int32)
    io = {"q": torch.zeros((B, H * G, D), dtype=torch.bfloat16, device=cuda), "lens": torch.zeros(B, dtype=torch.int32, device=cuda),
          "sel": torch.zeros((B, H, budget), dtype=torch.int32, device=cuda), "sl": torch.zeros((B, H), dtype=torch.int32, device=cuda)}
    db, ds, dt = bounds.to(cuda), scales.to(cuda), table.to(cuda)

    def call(stream=None):
        kv.nvfp4_kv_select_pages(kv.Layout(H, D, T), io["q"], db, ds, dt, io["lens"], io["sel"], io["sl"], sink_pages=1,
                                 recent_pages=2, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for high in (maxp * T, 20 * T, 1, maxp * T):
        lens = torch.randint(0, high + 1, (B,), generator=g, dtype=torch.int32)
        q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)
        io["lens"].copy_(lens), io["q"].copy_(q)
        graph.replay()
        want = plain_steps.select(q.double().numpy(), bounds.numpy(), scales.double().numpy(), table.numpy(), lens.numpy(), T,
                                  budget, 1, 2)
        assert np.array_equal(io["sel"].cpu().numpy(), want[1]) and np.array_equal(io["sl"].cpu().numpy(), want[2])


def test_unwritten_bounds_only_cost_their_page(kv, cuda):
    """Bounds and scales of NaN and infinity (never written): every id selected is still one of the
    sequence's pages, in order, and the pages with finite bounds keep their order among themselves."""
    D, T, H = 64, 16, 1
    bounds, scales, g = some_pages(60, H, D, 31)
    table = torch.randperm(60, generator=g).to(torch.int32)[None]
    bad = torch.tensor([5, 17, 40])
    scales[table[0, bad].long()] = torch.tensor([float("nan"), float("inf"), float("-inf")])[:, None]
    bounds[table[0, bad].long()] = -128
    q = torch.randn((1, 2, D), generator=g).to(torch.bfloat16)
    index, sel, sl, scores = selection(kv, cuda, q, bounds, scales, table, torch.tensor([960], dtype=torch.int32), H, T, 12, 1, 1)
    assert (np.diff(index[0, 0]) > 0).all() and index[0, 0, 0] == 0 and index[0, 0, -1] == 59
    assert np.array_equal(sel[0, 0], table[0].numpy()[index[0, 0]]) and sl[0, 0] == 12 * T
    kept = [i for i in index[0, 0] if i not in bad]
    left = [i for i in range(1, 59) if i not in kept and i not in bad]
    assert min(scores[0, 0, kept]) >= max(scores[0, 0, left])


# ------------------------------------------------------------------------------------ attention

class Cache:
    def __init__(self, dev, P, H, T, D, seed, scale=(0x28, 0x39)):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dev, self.H, self.T, self.D = g, dev, H, T, D
        self.kd, self.vd = rand_u8((P, H, T, D // 2), g), rand_u8((P, H, T // 2, D), g)
        self.ks, self.vs = rand_u8((P, H, T, D // 16), g, *scale), rand_u8((P, H, T // 2, D // 16, 2), g, *scale)
        self.gk, self.gv = 0.8, 0.6
        self.sm = 1 / np.sqrt(D)

    def run(self, kv, q, table, lens, status=None, workspace=None, stream=None):
        dev = self.dev
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
        lse = torch.full(q.shape[:2], float("nan"), device=dev)
        kv.nvfp4_paged_sparse_decode_attention(
            kv.Layout(self.H, self.D, self.T), q.to(dev), self.kd.to(dev), self.ks.to(dev),
            torch.tensor([self.gk], device=dev), self.vd.to(dev), self.vs.to(dev), torch.tensor([self.gv], device=dev),
            table.to(dev), lens.to(dev), self.sm, out, lse=lse, status=status, workspace=workspace, stream=stream)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), lse.cpu().numpy()

    def want(self, q, table, lens):
        return plain_steps.attend(q.double().numpy(), self.kd.numpy(), self.ks.numpy(), self.vd.numpy(), self.vs.numpy(),
                                  np.float32(self.gk), np.float32(self.gv), table.numpy(), lens.numpy(), self.T, self.sm)

    def check(self, got, want):
        (out, lse), (wout, wlse) = got, want
        assert np.isfinite(out).all()
        a = np.abs(wout)
        half = np.where(a > 0, 2.0 ** (np.floor(np.log2(np.where(a > 0, a, 1.0))) - 8), 0.0)
        err = np.abs(out - wout)
        # out = bf16(x) with x within MAX_ABS of wout, MEAN_ABS in the mean: |out - wout| <= |bf16(x) - x| + |x - wout|, and
        # the first term is at most half a step of each value, so its mean at most that of the half steps. (It counts
        # where a pair has a single token: its output is a V value, not an average of many.)
        assert (err <= MAX_ABS + half).all() and err.mean() <= MEAN_ABS + half.mean(), (err.max(), err.mean())
        fin = np.isfinite(wlse)
        assert np.array_equal(fin, np.isfinite(lse)) and (lse[~fin] == -np.inf).all()
        assert not fin.any() or np.abs(lse[fin] - wlse[fin]).max() <= LSE_ABS

    def tables(self, B, most, lens):
        table = torch.randint(0, self.kd.shape[0], (B, self.H, most), generator=self.g, dtype=torch.int32)
        for b in range(B):
            for h in range(self.H):
                table[b, h, -(-max(0, int(lens[b, h])) // self.T):] = -1
        return table


def queries(c, B, G):
    return torch.randn((B, c.H * G, c.D), generator=c.g).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,G", [(16, 2, 1), (32, 3, 4), (64, 8, 8), (48, 1, 5), (128, 2, 3), (80, 2, 7)])
def test_attention_of_ragged_pairs(kv, cuda, D, T, H, G):
    """Every pair its own length (0, 1, a page, across pages, the whole table) and its own pages."""
    B, most = 5, max(3, 640 // T)
    c = Cache(cuda, 40, H, T, D, D + T)
    lens = torch.randint(0, most * T + 1, (B, H), generator=c.g, dtype=torch.int32)
    lens[0, 0], lens[1, 0], lens[2, 0], lens[3, H - 1], lens[4, 0] = 0, 1, T, T + 1, most * T
    q, table = queries(c, B, G), c.tables(B, most, lens)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    c.check(c.run(kv, q, table, lens, status), c.want(q, table, lens))
    assert status.item() == 0


@pytest.mark.parametrize("B,H,most,low", [(1, 1, 1, 16), (1, 1, 400, 6400), (1, 8, 64, 900), (300, 4, 3, 0), (2, 2, 150, 0),
                                            (500, 8, 9, 0), (240, 8, 6, 90), (61, 7, 40, 500), (60, 8, 33, 0)])
def test_attention_of_few_and_many_pairs(kv, cuda, B, H, most, low):
    """One pair over one page or split over every SM, 1200 short pairs; more pairs than the 1824 warps, and
    pairs whose runs of their own would be more than the warps (runs then cross pairs)."""
    T, D, G = 16, 128, 4 if B < 100 else 1
    c = Cache(cuda, 90, H, T, D, B + H)
    lens = torch.randint(low, most * T + 1, (B, H), generator=c.g, dtype=torch.int32)
    q, table = queries(c, B, G), c.tables(B, most, lens)
    c.check(c.run(kv, q, table, lens), c.want(q, table, lens))


@pytest.mark.parametrize("B,H,G,D,T,pages", [
    (1, 8, 4, 128, 64, 64), (2, 4, 8, 256, 16, 70), (1, 5, 1, 64, 32, 300),   # clusters of 8 CTAs a pair
    (4, 5, 3, 128, 16, 150), (8, 4, 8, 64, 64, 40),                            # of 4
    (8, 8, 2, 128, 64, 30), (12, 5, 7, 256, 32, 33),                           # of 2
    (40, 3, 5, 128, 16, 70), (40, 8, 4, 128, 64, 9), (110, 8, 1, 64, 16, 21),  # one CTA for 1, 2 or 3, and 6 pairs
    (20, 8, 1, 64, 64, 64), (19, 8, 8, 128, 16, 90), (290, 8, 2, 256, 16, 3),  # runs over all pairs
])
@pytest.mark.parametrize("lengths", ["full", "ragged", "one long"])
def test_attention_however_it_is_cut(kv, cuda, B, H, G, D, T, pages, lengths):
    """The same result for every way to cut the pairs: all of full length, ragged with empty pairs, and one long
    among short ones, each with some pages outside the pool."""
    c = Cache(cuda, 50, H, T, D, B + pages)
    full = torch.full((B, H), pages * T, dtype=torch.int32)
    lens = full.clone()
    if lengths != "full":
        lens = torch.randint(0, pages * T + 1 if lengths == "ragged" else T + 2, (B, H), generator=c.g, dtype=torch.int32)
        lens[B // 2, 0] = pages * T
        lens[0, H - 1] = 0
    q, table = queries(c, B, G), c.tables(B, pages, lens)
    bad = torch.rand(table.shape, generator=c.g) < 0.02
    table = torch.where(bad, 50, table)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    n = kv.nvfp4_paged_sparse_decode_workspace_size(kv.Layout(H, D, T), B, H * G, pages)
    w = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda)
    got = c.run(kv, q, table, lens, status, w)
    c.check(got, c.want(q, table, lens))
    read = bad & (torch.arange(pages) * T < lens[..., None])
    assert status.item() == (kv.STATUS_PAGE_OOB if bool(read.any()) else 0)
    again = c.run(kv, q, table, lens, status, w)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("B,H,G,D,T,pages", [(1, 8, 4, 128, 64, 64), (4, 5, 3, 128, 16, 150), (8, 8, 2, 128, 64, 30),
                                             (40, 3, 5, 64, 16, 70), (20, 8, 1, 64, 64, 64)])
def test_attention_captured_and_replayed(kv, cuda, B, H, G, D, T, pages):
    """One graph of two calls that share a workspace, replayed while the lengths change what the pairs are cut into."""
    c = Cache(cuda, 40, H, T, D, B * pages)
    pool = [t.to(cuda) for t in (c.kd, c.ks, c.vd, c.vs)]
    g = [torch.tensor([x], device=cuda) for x in (c.gk, c.gv)]
    lay = kv.Layout(H, D, T)
    full = torch.full((B, H), pages * T, dtype=torch.int32)
    q = [queries(c, B, G) for _ in range(2)]
    table = torch.randint(0, 40, (B, H, pages), generator=c.g, dtype=torch.int32)
    dq, dt, dl = [x.to(cuda) for x in q], table.to(cuda), full.to(cuda)
    out = [torch.zeros_like(x) for x in dq]
    lse = [torch.zeros(x.shape[:2], device=cuda) for x in dq]
    w = torch.empty(kv.nvfp4_paged_sparse_decode_workspace_size(lay, B, H * G, pages), dtype=torch.uint8, device=cuda)

    def calls():
        for i in range(2):
            kv.nvfp4_paged_sparse_decode_attention(lay, dq[i], pool[0], pool[1], g[0], pool[2], pool[3], g[1], dt, dl, c.sm,
                                                   out[i], lse=lse[i], workspace=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    short = torch.randint(0, T + 2, (B, H), generator=c.g, dtype=torch.int32)
    short[B // 2, 0] = pages * T
    for lens in (full, short, torch.zeros_like(full), torch.full_like(full, 1), short, full):
        dl.copy_(lens)
        for o, s in zip(out, lse):
            o.fill_(float("nan"))
            s.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            c.check((out[i].float().cpu().numpy(), lse[i].cpu().numpy()), c.want(q[i], table, lens))


def test_all_pairs_empty(kv, cuda):
    c = Cache(cuda, 4, 3, 16, 64, 0)
    lens = torch.zeros((2, 3), dtype=torch.int32)
    out, lse = c.run(kv, queries(c, 2, 2), c.tables(2, 5, lens), lens)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_garbage_past_the_end_is_not_read(kv, cuda):
    """NaN scales in the tokens past a pair's end, ids outside the pool past its pages."""
    B, H, T, D, G = 3, 2, 32, 128, 4
    c = Cache(cuda, 30, H, T, D, 3)
    lens = torch.tensor([[33, 1], [65, 127], [95, 31]], dtype=torch.int32)
    table = torch.randperm(30, generator=c.g).to(torch.int32)[:24].view(B, H, 4).clone()
    q = queries(c, B, G)
    clean = c.run(kv, q, table, lens)
    for b in range(B):
        for h in range(H):
            n = int(lens[b, h])
            last, t = int(table[b, h, (n - 1) // T]), (n - 1) % T + 1
            c.ks[last, h, t:] = 0x7F
            for i in range(t, T):
                c.vs[last, h, i // 2, :, i % 2] = 0x7F
            c.kd[last, h, t:] = 0x77
            table[b, h, -(-n // T):] = 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = c.run(kv, q, table, lens, status)
    assert status.item() == 0
    assert np.array_equal(got[0], clean[0]) and np.array_equal(got[1], clean[1])
    c.check(got, c.want(q, table, lens))


def test_bad_pages_and_lengths(kv, cuda):
    B, H, T, D, G = 3, 2, 16, 64, 2
    c = Cache(cuda, 20, H, T, D, 4)
    lens = torch.tensor([[40, 80], [80, 16], [70, 64]], dtype=torch.int32)
    table, q = c.tables(B, 5, lens), queries(c, B, G)
    table[0, 1, 2], table[1, 1, 0], table[2, 0, 4] = 20, -3, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    c.check(c.run(kv, q, table, lens, status), c.want(q, table, lens))
    assert status.item() == kv.STATUS_PAGE_OOB
    lens[0, 0], lens[2, 1] = -1, 81
    status.zero_()
    c.check(c.run(kv, q, table, lens, status), c.want(q, table, lens))
    assert status.item() == kv.STATUS_PAGE_OOB | kv.STATUS_BAD_SEQ_LEN


def test_a_page_listed_twice_counts_twice(kv, cuda):
    c = Cache(cuda, 5, 1, 16, 64, 5)
    lens = torch.tensor([[48]], dtype=torch.int32)
    table, q = torch.tensor([[[2, 2, 3]]], dtype=torch.int32), queries(c, 1, 2)
    c.check(c.run(kv, q, table, lens), c.want(q, table, lens))


def test_large_scores_and_equal_keys(kv, cuda):
    """Scores in the thousands (one key takes everything) and keys that are all alike."""
    c = Cache(cuda, 12, 2, 16, 128, 6, scale=(0x50, 0x60))
    lens = torch.tensor([[190, 77]], dtype=torch.int32)
    table, q = c.tables(1, 12, lens), queries(c, 1, 3)
    c.gv = 0.001
    c.check(c.run(kv, q, table, lens), c.want(q, table, lens))
    c.kd[:], c.ks[:] = 0x22, 0x38
    c.check(c.run(kv, q, table, lens), c.want(q, table, lens))


def test_equals_the_dense_decode(kv, cuda):
    """Every head of a sequence given the whole sequence: the dense call's result (in its tolerance)."""
    B, H, T, D, G = 3, 4, 64, 128, 4
    c = Cache(cuda, 60, H, T, D, 7)
    lens = torch.tensor([640, 1, 333], dtype=torch.int32)
    table = torch.randperm(60, generator=c.g).to(torch.int32)[:30].view(3, 10)
    q = queries(c, B, G)
    per, pl = table[:, None].expand(B, H, 10).contiguous(), lens[:, None].expand(B, H).contiguous()
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=cuda)
    lse = torch.empty(q.shape[:2], device=cuda)
    kv.nvfp4_paged_decode_attention(kv.Layout(H, D, T), q.to(cuda), c.kd.to(cuda), c.ks.to(cuda),
                                    torch.tensor([c.gk], device=cuda), c.vd.to(cuda), c.vs.to(cuda),
                                    torch.tensor([c.gv], device=cuda), table.to(cuda), lens.to(cuda), c.sm, out, lse=lse)
    got = c.run(kv, q, per, pl)
    c.check(got, (out.double().cpu().numpy(), lse.double().cpu().numpy()))
    c.check(got, c.want(q, per, pl))


@pytest.mark.parametrize("fill", [0xFF, "random"])
def test_workspace_needs_no_clearing(kv, cuda, fill):
    B, H, T, D, G = 2, 2, 16, 128, 4
    c = Cache(cuda, 50, H, T, D, 8)
    lens = torch.tensor([[800, 640], [16, 790]], dtype=torch.int32)
    table, q = c.tables(B, 50, lens), queries(c, B, G)
    n = kv.nvfp4_paged_sparse_decode_workspace_size(kv.Layout(H, D, T), B, H * G, 50)
    w = torch.zeros(n, dtype=torch.uint8, device=cuda)
    clean = c.run(kv, q, table, lens, workspace=w)
    w = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda) if fill == 0xFF else rand_u8((n,), c.g).to(cuda)
    for _ in range(2):
        got = c.run(kv, q, table, lens, workspace=w)
        assert np.array_equal(got[0], clean[0]) and np.array_equal(got[1], clean[1])
    c.check(got, c.want(q, table, lens))


def test_pages_past_32_bit_byte_offsets(kv, cuda):
    """Bounds, selection and attention on pages whose codes lie past 2^32 bytes."""
    H, D, T, G = 8, 256, 128, 2
    P = (1 << 32) // (H * T * D // 2) + 8
    far = [P - 1, P - 5, 0, P - 2, 3, P - 8]
    small = Cache(cuda, len(far), H, T, D, 12)
    big = [torch.zeros((P, *t.shape[1:]), dtype=torch.uint8, device=cuda) for t in (small.kd, small.ks, small.vd, small.vs)]
    for t, s in zip(big, (small.kd, small.ks, small.vd, small.vs)):
        t[far] = s.to(cuda)
    lay, ids = kv.Layout(H, D, T), torch.tensor(far, dtype=torch.int32, device=cuda)
    bounds, scales = torch.zeros((P, H, 2, D), dtype=torch.int8, device=cuda), torch.zeros((P, H), device=cuda)
    kv.nvfp4_kv_page_bounds(lay, big[0], big[1], bounds, scales, page_ids=ids)
    q, lens = queries(small, 1, G), torch.tensor([5 * T + 9], dtype=torch.int32)
    want = plain_steps.select(q.double().numpy(), bounds[far].cpu().numpy(), scales[far].double().cpu().numpy(),
                              np.arange(6)[None], lens.numpy(), T, 4, 1, 1)
    table = torch.full((1, H, 4), 5, dtype=torch.int32, device=cuda)
    sl = torch.zeros((1, H), dtype=torch.int32, device=cuda)
    kv.nvfp4_kv_select_pages(lay, q.to(cuda), bounds, scales, ids[None].contiguous(), lens.to(cuda), table, sl)
    assert np.array_equal(table.cpu().numpy(), np.array(far)[want[1]])
    out, lse = torch.empty((1, H * G, D), dtype=torch.bfloat16, device=cuda), torch.empty((1, H * G), device=cuda)
    g = [torch.tensor([x], device=cuda) for x in (small.gk, small.gv)]
    kv.nvfp4_paged_sparse_decode_attention(lay, q.to(cuda), big[0], big[1], g[0], big[2], big[3], g[1], table, sl, small.sm,
                                           out, lse=lse)
    ref = small.want(q, torch.from_numpy(want[1]), torch.from_numpy(want[2]))
    small.check((out.float().cpu().numpy(), lse.cpu().numpy()), ref)


# ------------------------------------------------------------------------------------ together

class Steps:
    """Sequences that decode step by step: append, bounds of the pages that became full, selection,
    attention; on the GPU and in the plain forms."""

    def __init__(self, kv, cuda, B=3, H=2, G=3, D=64, T=16, maxp=20, budget=6, seed=0):
        self.kv, self.dev = kv, cuda
        self.B, self.H, self.G, self.D, self.T, self.maxp, self.budget = B, H, G, D, T, maxp, budget
        self.g = torch.Generator().manual_seed(seed)
        P = self.P = B * maxp
        self.table = torch.randperm(P, generator=self.g).to(torch.int32).view(B, maxp)
        z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
        self.host = {"kd": z(P, H, T, D // 2), "ks": z(P, H, T, D // 16), "vd": z(P, H, T // 2, D), "vs": z(P, H, T // 2, D // 16, 2)}
        self.pool = {n: t.to(cuda) for n, t in self.host.items()}
        self.host = {n: t.numpy() for n, t in self.host.items()}
        self.hb, self.hs = np.zeros((P, H, 2, D), np.int8), np.zeros((P, H), np.float32)
        ang = torch.arange(1000, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        dev = cuda
        e = lambda s, dt: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
        Hq = H * G
        self.io = {"q": e((B, Hq, D), torch.bfloat16), "k": e((B, H, D), torch.bfloat16), "v": e((B, H, D), torch.bfloat16),
                   "slots": e((B,), torch.int64), "positions": e((B,), torch.int32), "full": e((B,), torch.int32),
                   "lens": e((B,), torch.int32), "q_out": e((B, Hq, D), torch.bfloat16),
                   "bounds": e((P, H, 2, D), torch.int8), "bound_scales": e((P, H), torch.float32),
                   "sel": e((B, H, budget), torch.int32), "sl": e((B, H), torch.int32),
                   "out": e((B, Hq, D), torch.bfloat16), "lse": e((B, Hq), torch.float32), "status": e((1,), torch.int32)}
        self.rot = kv.Rotary(kv.ROTARY_HALVES, 0, D, self.cos_sin.to(dev))
        self.scale = [torch.tensor([x], device=dev) for x in (0.002, 0.001)]
        self.dtable = self.table.to(dev)
        lay = self.lay = kv.Layout(H, D, T)
        self.ws = e((kv.nvfp4_paged_sparse_decode_workspace_size(lay, B, Hq, budget),), torch.uint8)

    def launch(self):
        kv, io, p = self.kv, self.io, self.pool
        kv.nvfp4_kv_append(self.lay, io["k"], io["v"], io["slots"], p["kd"], p["ks"], p["vd"], p["vs"], q=io["q"],
                           q_out=io["q_out"], rotary=self.rot, positions=io["positions"], k_global_scale=self.scale[0],
                           v_global_scale=self.scale[1], status=io["status"])
        kv.nvfp4_kv_page_bounds(self.lay, p["kd"], p["ks"], io["bounds"], io["bound_scales"], page_ids=io["full"],
                                status=io["status"])
        kv.nvfp4_kv_select_pages(self.lay, io["q_out"], io["bounds"], io["bound_scales"], self.dtable, io["lens"], io["sel"],
                                 io["sl"], sink_pages=1, recent_pages=2, status=io["status"])
        kv.nvfp4_paged_sparse_decode_attention(self.lay, io["q_out"], p["kd"], p["ks"], self.scale[0], p["vd"], p["vs"],
                                               self.scale[1], io["sel"], io["sl"], 0.125, io["out"], lse=io["lse"],
                                               workspace=self.ws, status=io["status"])

    def feed(self, lens):
        """New rows for tokens lens[b] (a sequence at -1 is idle); returns the host copies."""
        B, H, D, T = self.B, self.H, self.D, self.T
        x = {"q": torch.randn((B, H * self.G, D), generator=self.g).to(torch.bfloat16),
             "k": torch.randn((B, H, D), generator=self.g).to(torch.bfloat16),
             "v": torch.randn((B, H, D), generator=self.g).to(torch.bfloat16)}
        n = torch.tensor(lens)
        page = self.table.gather(1, (n.clamp(min=0) // T)[:, None])[:, 0].long()
        x["slots"] = torch.where(n >= 0, page * T + n % T, -1)
        x["positions"] = n.clamp(min=0).to(torch.int32)
        x["full"] = torch.where((n >= 0) & (n % T == T - 1), page, -1).to(torch.int32)
        x["lens"] = (n + 1).to(torch.int32)
        for name, t in x.items():
            self.io[name].copy_(t)
        return x

    def plain(self, x):
        f = lambda t: t.double().numpy()  # noqa: E731
        qs, _, _ = plain_steps.append(self.host, f(x["k"]), f(x["v"]), x["slots"].numpy(), self.T, np.float32(0.002),
                                      np.float32(0.001), ("halves", 0, self.D, self.cos_sin.numpy()), x["positions"].numpy(),
                                      f(x["q"]))
        for page in x["full"].tolist():
            if page >= 0:
                self.hb[page, :, 0], self.hb[page, :, 1], self.hs[page] = plain_steps.page_bounds(
                    self.host["kd"][page], self.host["ks"][page], self.T)
        q = self.io["q_out"].double().cpu().numpy()
        for b, w in enumerate(qs):
            if w is not None:
                assert np.array_equal(torch.from_numpy(w).float().to(torch.bfloat16).double().numpy(), q[b])
        index, sel, sl, _ = plain_steps.select(q, self.hb, self.hs.astype(np.float64), self.table.numpy(), x["lens"].numpy(), self.T, self.budget, 1, 2)
        assert np.array_equal(self.io["sel"].cpu().numpy(), sel) and np.array_equal(self.io["sl"].cpu().numpy(), sl)
        for n, t in self.pool.items():
            assert np.array_equal(t.cpu().numpy(), self.host[n]), n
        out, lse = plain_steps.attend(q, self.host["kd"], self.host["ks"], self.host["vd"], self.host["vs"], np.float32(0.002),
                                      np.float32(0.001), sel, sl, self.T, 0.125)
        got = self.io["out"].double().cpu().numpy()
        a = np.abs(out)
        half = np.where(a > 0, 2.0 ** (np.floor(np.log2(np.where(a > 0, a, 1.0))) - 8), 0.0)
        assert (np.abs(got - out) <= MAX_ABS + half).all()
        fin = np.isfinite(lse)
        glse = self.io["lse"].cpu().numpy()
        assert np.array_equal(fin, np.isfinite(glse)) and np.abs(glse[fin] - lse[fin]).max() <= LSE_ABS
        assert self.io["status"].item() == 0


def test_decode_steps_together(kv, cuda):
    """150 steps of three sequences that start apart (one joins late, one pauses)."""
    s = Steps(kv, cuda)
    lens = [0, -1, 0]
    for i in range(150):
        if i == 40:
            lens[1] = 0
        now = [n if not (b == 2 and 60 <= i < 70) else -1 for b, n in enumerate(lens)]
        x = s.feed(now)
        if i == 40:
            assert now[1] == 0
        for b in range(3):                       # an idle sequence keeps its length
            if now[b] < 0:
                x["lens"][b] = max(0, lens[b])
        s.io["lens"].copy_(x["lens"])
        s.launch()
        if i % 13 == 0 or i in (15, 16, 41, 65, 149):
            s.plain(x)
        else:                                    # keep the plain cache up to date
            f = lambda t: t.double().numpy()  # noqa: E731
            plain_steps.append(s.host, f(x["k"]), f(x["v"]), x["slots"].numpy(), s.T, np.float32(0.002), np.float32(0.001),
                               ("halves", 0, s.D, s.cos_sin.numpy()), x["positions"].numpy(), f(x["q"]))
            for page in x["full"].tolist():
                if page >= 0:
                    s.hb[page, :, 0], s.hb[page, :, 1], s.hs[page] = plain_steps.page_bounds(s.host["kd"][page], s.host["ks"][page], s.T)
        lens = [n + 1 if now[b] >= 0 else n for b, n in enumerate(lens)]


def test_steps_captured_in_two_graphs_that_share_a_workspace(kv, cuda):
    """Two layers' steps captured in two graphs over one workspace, replayed in turn."""
    one, two = Steps(kv, cuda, seed=1), Steps(kv, cuda, seed=2)
    two.ws = one.ws
    graphs = []
    for s in (one, two):
        s.feed([-1, -1, -1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.launch()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.launch()
        graphs.append(g)
    for i in range(40):
        for s, g in zip((one, two) if i % 2 else (two, one), graphs if i % 2 else graphs[::-1]):
            x = s.feed([i, i, i])
            g.replay()
            torch.cuda.synchronize()
            s.plain(x)


def test_two_calls_at_once_on_two_streams(kv, cuda):
    """Two selections and attentions on two streams, each with a workspace of its own."""
    B, H, T, D, G = 4, 4, 16, 128, 2
    c = Cache(cuda, 100, H, T, D, 20)
    lens = torch.randint(1, 60 * T, (B, H), generator=c.g, dtype=torch.int32)
    table = c.tables(B, 60, lens)
    qs = [queries(c, B, G) for _ in range(2)]
    alone = [c.run(kv, q, table, lens) for q in qs]
    dev = {n: getattr(c, n).to(cuda) for n in ("kd", "ks", "vd", "vs")}
    gs = [torch.tensor([x], device=cuda) for x in (c.gk, c.gv)]
    dt, dl, dq = table.to(cuda), lens.to(cuda), [q.to(cuda) for q in qs]
    outs = [torch.zeros(q.shape, dtype=torch.bfloat16, device=cuda) for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    lay = kv.Layout(H, D, T)
    ws = [torch.empty(kv.nvfp4_paged_sparse_decode_workspace_size(lay, B, H * G, 60), dtype=torch.uint8, device=cuda) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, o, w, s in zip(dq, outs, ws, streams):
            kv.nvfp4_paged_sparse_decode_attention(lay, q, dev["kd"], dev["ks"], gs[0], dev["vd"], dev["vs"], gs[1], dt, dl, c.sm, o,
                                                   workspace=w, stream=s)
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert np.array_equal(o.float().cpu().numpy(), a[0])


def test_binding_refuses_on_the_gpu(kv, cuda):
    lay = kv.Layout(8, 128, 64)
    z = lambda dt, *s: torch.zeros(s, dtype=dt, device=cuda)  # noqa: E731
    u8, i8, i32, f32, bf = torch.uint8, torch.int8, torch.int32, torch.float32, torch.bfloat16
    kd, ks, bo, sc = z(u8, 2, 8, 64, 64), z(u8, 2, 8, 64, 8), z(i8, 2, 8, 2, 128), z(f32, 2, 8)
    for bad in ((kd[..., :32], ks, bo, sc, {}), (kd, ks[..., :4].contiguous(), bo, sc, {}), (kd, ks, bo[:1], sc, {}),
                (kd, ks, bo.to(u8), sc, {}), (kd, ks, bo, sc[:, :7], {}), (kd, ks, bo, sc.double(), {}),
                (kd, ks, bo, sc, dict(page_ids=z(i32, 3), page_tokens=z(i32, 2))), (kd, ks, bo, sc, dict(page_ids=z(torch.int64, 3))),
                (kd, ks, bo.cpu(), sc, {})):
        with pytest.raises(ValueError):
            kv.nvfp4_kv_page_bounds(lay, *bad[:4], **bad[4])
    q = z(bf, 3, 16, 128)
    good = dict(q=q, bounds=bo, bound_scales=sc, page_table=z(i32, 3, 5), seq_lens=z(i32, 3), sel_page_table=z(i32, 3, 8, 2),
                sel_lens=z(i32, 3, 8))
    kv.nvfp4_kv_select_pages(lay, **good)
    for bad in (dict(q=q[..., :64]), dict(q=q.float()), dict(seq_lens=z(i32, 2)), dict(sel_lens=z(i32, 8)),
                dict(sel_page_table=z(i32, 3, 7, 2)), dict(page_table=z(torch.int64, 3, 5)), dict(scores=z(f32, 3, 8, 4)),
                dict(sel_index=z(i32, 3, 8, 3)), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(bounds=bo[:1])):
        with pytest.raises(ValueError):
            kv.nvfp4_kv_select_pages(lay, **{**good, **bad})
    with pytest.raises(kv.NVFP4KVError, match="INVALID"):
        kv.nvfp4_kv_select_pages(lay, **good, sink_pages=2)
    g = z(f32, 1)
    pool = [kd, ks, g, z(u8, 2, 8, 32, 128), z(u8, 2, 8, 32, 8, 2), g]
    kv.nvfp4_paged_sparse_decode_attention(lay, q, *pool, z(i32, 3, 8, 2), z(i32, 3, 8), 0.1, torch.zeros_like(q))
    for tab, ln, out, kw in ((z(i32, 3, 8, 2), z(i32, 3, 7), q, {}), (z(i32, 3, 7, 2), z(i32, 3, 8), q, {}),
                             (z(i32, 3, 8, 2), z(i32, 3, 8), q.half(), {}), (z(i32, 3, 8, 2), z(i32, 3, 8), q, dict(lse=z(f32, 3, 15))),
                             (z(i32, 3, 8, 2), z(i32, 3, 8), q, dict(workspace=torch.zeros(1 << 20, dtype=u8)))):
        with pytest.raises(ValueError):
            kv.nvfp4_paged_sparse_decode_attention(lay, q, *pool, tab, ln, 0.1, out, **kw)
    with pytest.raises(kv.NVFP4KVError, match="WORKSPACE"):
        kv.nvfp4_paged_sparse_decode_attention(lay, q, *pool, z(i32, 3, 8, 2), z(i32, 3, 8), 0.1, torch.zeros_like(q),
                                               workspace=z(u8, 64))
