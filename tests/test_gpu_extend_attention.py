"""The extend attention against a 64-bit form, within bounds derived from its roundings (plain_windows.check)."""
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


class Chunk(Cache):
    """Sequences of `lens` tokens whose last `new` are the chunk's rows, with padding rows behind them."""

    def __init__(self, dev, lens, new, H, T, D, G, padding=0, wide=False, **kw):
        # (a page that only the last token's window hides is still needed by the first row)
        super().__init__(dev, "fp8", lens, H, T, D, G, drop=False, **kw)
        self.new = list(new)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.rows = int(self.starts[-1]) + padding
        x = torch.randn((self.rows, (H * G + 2) * D), generator=self.g).to(torch.bfloat16)
        self.qkv = x.to(dev)
        self.q = x[:, :H * G * D].view(self.rows, H * G, D)
        self.q_dev = self.qkv[:, :H * G * D].view(self.rows, H * G, D) if wide else self.q.contiguous().to(dev)
        if self.window:  # pages that no row sees have been given back
            for b, n in enumerate(self.lens):
                first = n - self.new[b] - self.window + 1
                for j in range(-(-n // T)):
                    if (j + 1) * T <= first and j * T >= self.sinks:
                        self.table[b, j] = -1 if j % 2 else 2 ** 31 - 1

    def run(self, kv, starts=None, lens=None, fill=float("nan"), out=None, **kw):
        i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=self.dev)  # noqa: E731
        hq = self.H * self.G
        out = torch.full((self.rows, hq, self.D), fill, dtype=torch.bfloat16, device=self.dev) if out is None else out
        lse = torch.full((self.rows, hq), fill, device=self.dev)
        pools, scales = self.fp8()
        kv.nvfp4_paged_extend_attention(self.layout(kv), self.q_dev, *pools, self.table.to(self.dev), i(self.lens if lens is None else lens),
                                        i(self.starts if starts is None else starts), self.sm, out, lse=lse, window=self.window,
                                        sink_tokens=self.sinks, **scales, **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, got, some=None):
        """Every row, or of each sequence at most `some`, its first and last among them; padding as it was."""
        out, lse = got
        assert np.isnan(out[self.starts[-1]:]).all() and np.isnan(lse[self.starts[-1]:]).all()
        assert np.isfinite(out[:self.starts[-1]]).all()
        G = self.G
        for b, n in enumerate(self.lens):
            m = self.new[b]
            if m == 0:
                continue
            at = np.arange(m) if some is None or m <= some else np.unique(np.linspace(0, m - 1, some).astype(int))
            rows = self.starts[b] + at
            for h in range(self.H):
                k, v, ok = self.tokens(b, h)
                here = np.repeat(plain_windows.visible(n - m + at, n, self.window, self.sinks) & ok, G, 0)
                heads = slice(h * G, (h + 1) * G)
                plain_windows.check((out[rows, heads].reshape(-1, self.D), lse[rows, heads].reshape(-1)),
                                    self.q[rows, heads].double().numpy().reshape(-1, self.D), k, v, here, self.sm, self.vmax(), blocks=True)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (256, 4), (64, 1), (128, 8), (256, 3), (128, 7)])
def test_one_small_chunk(kv, cuda, D, G):
    """A chunk of a few tokens without a prefix, one behind one, and single rows."""
    for lens, new in (([1], [1]), ([5], [5]), ([37], [3]), ([300], [1])):
        c = Chunk(cuda, lens, new, 1, 16, D, G, seed=G)
        c.check(c.run(kv))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [16, 48, 64, 128])
def test_ragged_chunks(kv, cuda, D, T):
    """Prompts, chunks behind prefixes, decode rows, sequences without rows, empty ones, padding rows."""
    for H, G, blocks in ((2, 4, True), (3, 1, False), (1, 6, True)):
        lens, new = [200, 0, 1, 130, 77, 300, 64, 5], [200, 0, 1, 2, 0, 150, 64, 5]
        c = Chunk(cuda, lens, new, H, T, D, G, padding=5, seed=T + H, blocks=blocks)
        c.check(c.run(kv))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_windows(kv, cuda, D):
    """Windows and first tokens that end inside tiles and pages; windows of one token; wider than the sequence."""
    for T, window, sinks in ((16, 1, 0), (64, 100, 4), (32, 33, 140), (64, 64, 64), (48, 500, 1), (128, 5000, 9), (16, 257, 300)):
        c = Chunk(cuda, [700, 1000, 1, 90, 400], [130, 1, 1, 90, 0], 2, T, D, 4, window=window, sinks=sinks, seed=window, padding=1)
        c.check(c.run(kv), some=60)


@pytest.mark.parametrize("D,H,G", [(64, 2, 8), (128, 2, 4), (256, 1, 2)])
def test_long_prefixes_are_cut_and_joined(kv, cuda, D, H, G):
    """Few units over all SMs, a workspace of garbage; the same result again."""
    for lens, new in (([20000], [40]), ([9000, 12000, 64], [1, 300, 64]), ([5000], [1])):
        c = Chunk(cuda, lens, new, H, 64, D, G, seed=len(lens))
        size = kv.nvfp4_paged_extend_attention_workspace_size(c.layout(kv), len(lens), H * G)
        ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=cuda)
        first = c.run(kv, workspace=ws)
        c.check(first, some=24)
        again = c.run(kv, workspace=ws.random_(0, 256))
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_a_long_prompt(kv, cuda):
    c = Chunk(cuda, [6000], [6000], 2, 64, 128, 4, seed=1)
    c.check(c.run(kv), some=40)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_projection(kv, cuda, D):
    """Strided queries and outputs; what lies beside the outputs is left as it was."""
    c = Chunk(cuda, [100, 260], [50, 9], 2, 16, D, 4, wide=True, padding=2)
    whole = torch.full((c.rows, 8 * D + 64), 7.0, dtype=torch.bfloat16, device=cuda)
    out = whole[:, :8 * D].view(c.rows, 8, D)
    out.fill_(float("nan"))
    c.check(c.run(kv, out=out))
    assert bool((whole[:, 8 * D:] == 7).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_pages_lengths_and_rows(kv, cuda, D):
    """Ids outside the pool leave their tokens out, all that a row sees among them; lengths and rows out of range give 0 and
    -inf where the rows can be told, and touch nothing else."""
    c = Chunk(cuda, [200, 150, 40, 90], [60, 3, 20, 90], 2, 16, D, 2, window=120, sinks=20, seed=D)
    c.table[0, 12], c.table[0, 6], c.table[0, 0] = c.P, -1, 2 ** 31 - 1
    c.table[2, :] = -1
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = c.run(kv, status=status)
    c.check(got)
    assert status.item() == kv.STATUS_PAGE_OOB
    good = c.run(kv)
    for lens in ([200, 2, 40, 90], [200, -1, 40, 90], [200, c.maxp * 16 + 1, 40, 90], [200, 2 ** 31 - 1, 40, 90]):
        status.zero_()
        out, lse = c.run(kv, lens=lens, status=status)
        assert (out[60:63] == 0).all() and (lse[60:63] == -np.inf).all()
        assert status.item() & kv.STATUS_BAD_SEQ_LEN
        for rows in (slice(0, 60), slice(63, None)):
            assert np.array_equal(out[rows], good[0][rows]) and np.array_equal(lse[rows], good[1][rows])
    status.zero_()
    out, lse = c.run(kv, starts=[0, 60, 63, 83, 999], status=status)
    assert np.isnan(out[83:]).all() and np.array_equal(out[:83], good[0][:83]) and status.item() & kv.STATUS_BAD_SEQ_LEN
    for starts in ([-5, -4, -3, -2, -1], [0, -1, 0, -1, 0], [2 ** 31 - 1] * 5, [-2 ** 31, 2 ** 31 - 1, 0, 0, 0]):
        out, lse = c.run(kv, starts=starts)
        assert np.isnan(out).all() and np.isnan(lse).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_no_row_sees_may_be_anything(kv, cuda, D):
    """NaN bytes in the tokens before every row's window and behind the end, NaN scales of pages without a visible token."""
    c = Chunk(cuda, [170, 300, 37], [20, 7, 37], 1, 32, D, 4, window=40, sinks=3, seed=5)
    want = c.run(kv)
    for b, n in enumerate(c.lens):
        first = n - c.new[b] - 40 + 1
        for j in range(-(-n // 32)):
            page = int(c.table[b, j])
            if not 0 <= page < c.P:
                continue
            hidden = [j * 32 + t >= n or (j * 32 + t < first and j * 32 + t >= 3) for t in range(32)]
            for t in range(32):
                if hidden[t]:
                    c.k[page, :, t], c.v[page, :, t] = 0x7F, 0xFF
            if all(hidden):
                c.kb[page], c.vb[page] = float("nan"), float("inf")
    got = c.run(kv)
    assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])


def test_scores_of_any_size_and_a_negative_scale(kv, cuda):
    """Queries of 2^-60 to 2^8 times the usual in one chunk, zero queries, and a negative softmax scale."""
    c = Chunk(cuda, [150], [64], 1, 16, 64, 2, seed=2)
    f = 2.0 ** torch.linspace(-60, 8, 64).round()
    f[7] = 0
    c.q = (c.q.float() * f[:, None, None]).to(torch.bfloat16)
    c.q_dev = c.q.to(cuda)
    for sm in (c.sm, -c.sm, 0.0):
        c.sm = sm
        c.check(c.run(kv))


def test_agrees_with_the_decode(kv, cuda):
    """Single rows against the FP8 decode, each within its bound (its own test), here to the neighbouring BF16 value."""
    lens = [400, 64, 1, 1000]
    c = Chunk(cuda, lens, [1] * 4, 2, 16, 128, 4, seed=6)
    out, lse = c.run(kv)
    d = Cache.run(c, kv)
    assert np.abs(out - d[0]).max() <= 2.0 ** -7 * np.abs(out).max() and np.abs(lse - d[1]).max() < 1e-4


def test_captured_and_replayed_over_new_lengths(kv, cuda):
    """A graph whose replays see other lengths, rows and queries; results equal those of eager calls."""
    c = Chunk(cuda, [500, 900, 64], [200, 1, 64], 2, 64, 128, 4, seed=8)
    B, rows, hq = 3, 300, 8
    q = torch.zeros((rows, hq, 128), dtype=torch.bfloat16, device=cuda)
    lens, starts = (torch.zeros(n, dtype=torch.int32, device=cuda) for n in (B, B + 1))
    out, lse = torch.zeros_like(q), torch.zeros((rows, hq), device=cuda)
    pools, scales = c.fp8()
    table = c.table.to(cuda)
    ws = torch.empty(kv.nvfp4_paged_extend_attention_workspace_size(c.layout(kv), B, hq), dtype=torch.uint8, device=cuda)

    def step():
        kv.nvfp4_paged_extend_attention(c.layout(kv), q, *pools, table, lens, starts, c.sm, out, lse=lse, workspace=ws, **scales)
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n, m in (([500, 900, 64], [200, 1, 64]), ([499, 130, 0], [1, 130, 0]), ([100, 900, 33], [100, 160, 33])):
        q.copy_(torch.randn(q.shape, generator=c.g).to(torch.bfloat16))
        lens.copy_(torch.tensor(n)), starts.copy_(torch.tensor([0, *np.cumsum(m)]))
        out.fill_(float("nan")), lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        c.lens, c.new, c.starts, c.rows = n, m, np.concatenate([[0], np.cumsum(m)]), rows
        c.q = q.cpu()
        c.check((got[0].double().cpu().numpy(), got[1].double().cpu().numpy()), some=30)
        ws.random_(0, 256)
        step()
        assert torch.equal(out.nan_to_num(), got[0].nan_to_num()) and torch.equal(lse.nan_to_num(), got[1].nan_to_num())


def test_two_calls_at_once(kv, cuda):
    """Calls on two streams with workspaces of their own, and with scratch that the binding takes."""
    cs = [Chunk(cuda, [800, 90], [300, 90], 2, 64, 128, 4, seed=i) for i in range(2)]
    want = [c.run(kv) for c in cs]
    i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=cuda)  # noqa: E731
    args = []
    for c in cs:
        pools, scales = c.fp8()
        args.append((c.layout(kv), c.q_dev, *pools, c.table.to(cuda), i(c.lens), i(c.starts), c.sm, torch.empty_like(c.q_dev), scales))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for s, a in zip(streams, args):
            kv.nvfp4_paged_extend_attention(*a[:-1], stream=s, **a[-1])
    torch.cuda.synchronize()
    for w, a in zip(want, args):
        assert np.array_equal(w[0], a[-2].double().cpu().numpy())
