"""The decode attentions over FP8 pages and with a sliding window against a 64-bit form, within bounds derived from their
roundings (plain_windows.check)."""
import numpy as np
import pytest
import torch

import plain_steps
import plain_windows
from test_gpu_fp8_pages import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


class Cache:
    """Pages of one format on the host and the GPU, with page tables of which the pages that the window hides hold
    garbage ids: given back."""

    def __init__(self, dev, fmt, lens, H, T, D, G, window=0, sinks=0, seed=0, blocks=True, drop=True, maxp=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.dev, self.fmt, self.H, self.T, self.D, self.G = dev, fmt, H, T, D, G
        self.lens, self.window, self.sinks = list(lens), window, sinks
        B = len(self.lens)
        n = [-(-x // T) for x in self.lens]
        self.maxp = maxp or max(1, max(n) + 1)
        P = self.P = sum(n) + 3
        perm = torch.randperm(P, generator=g).tolist()
        self.table = torch.full((B, self.maxp), -123456789, dtype=torch.int32)
        for b in range(B):
            for j in range(n[b]):
                page = perm.pop()
                seen = not window or not drop or (j + 1) * T > self.lens[b] - window or j * T < sinks
                self.table[b, j] = page if seen else (2 ** 31 - 1 if j % 2 else -1)
        u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
        self.sm = float(np.float32(D ** -0.5))
        if fmt == "fp8":
            self.k, self.v = ((torch.randn((P, H, T, D), generator=g) * 112).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                              for _ in range(2))
            self.kb, self.vb = (((torch.rand((P, H), generator=g) + 0.5) / 100 * 2.0 ** torch.randint(-3, 4, (P, H), generator=g))
                                if blocks else None for _ in range(2))
            self.ks, self.vs = (torch.tensor([0.8]), torch.tensor([1.3])) if seed % 2 or not blocks else (None, None)
            if not blocks:
                self.ks, self.vs = self.ks / 100, self.vs / 100
        else:
            self.kd, self.vd = u(0, 256, P, H, T, D // 2), u(0, 256, P, H, T // 2, D)
            self.ksc, self.vsc = u(0x28, 0x39, P, H, T, D // 16), u(0x28, 0x39, P, H, T // 2, D // 16, 2)
            self.gk, self.gv = torch.tensor([0.8]), torch.tensor([0.6])
        self.q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)

    def layout(self, kv):
        return kv.Layout(self.H, self.D, self.T)

    def fp8(self, to=None):
        d = lambda t: None if t is None else t.to(to or self.dev)  # noqa: E731
        return [d(self.k), d(self.v)], dict(k_block_scales=d(self.kb), v_block_scales=d(self.vb), k_scale=d(self.ks), v_scale=d(self.vs))

    def run(self, kv, lens=None, **kw):
        d = lambda t: t.to(self.dev)  # noqa: E731
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device=self.dev)
        lse = torch.full(self.q.shape[:2], float("nan"), device=self.dev)
        lens = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32, device=self.dev)
        if self.fmt == "fp8":
            pools, scales = self.fp8()
            kv.nvfp4_paged_fp8_decode_attention(self.layout(kv), d(self.q), *pools, d(self.table), lens, self.sm, out, lse=lse,
                                                window=self.window, sink_tokens=self.sinks, **scales, **kw)
        else:
            kv.nvfp4_paged_window_decode_attention(self.layout(kv), d(self.q), d(self.kd), d(self.ksc), d(self.gk), d(self.vd),
                                                   d(self.vsc), d(self.gv), d(self.table), lens, self.sm, out, lse=lse,
                                                   window=self.window, sink_tokens=self.sinks, **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def tokens(self, b, h):
        """k, v [n, D] of a sequence and head in 64 bits (pages that were given back or are bad read as NaN), and which
        tokens have a page."""
        n = self.lens[b]
        if n == 0:
            return np.zeros((0, self.D)), np.zeros((0, self.D)), np.zeros(0, bool)
        ids = self.table[b, :-(-n // self.T)].numpy()
        ok = (ids >= 0) & (ids < self.P)
        at = np.where(ok, ids, 0)
        if self.fmt == "fp8":
            k, v = (plain_windows.FP8[t.numpy()[at, h]] for t in (self.k, self.v))
            for x, sb, s in ((k, self.kb, self.ks), (v, self.vb, self.vs)):
                if sb is not None:
                    x *= sb.double().numpy()[at, h][:, None, None]
                if s is not None:
                    x *= float(s.double())
        else:
            k = plain_steps.keys(self.kd.numpy()[at, h], self.ksc.numpy()[at, h]) * float(self.gk.double())
            v = values(self.vd.numpy()[at, h], self.vsc.numpy()[at, h]) * float(self.gv.double())
        return k.reshape(-1, self.D)[:n], v.reshape(-1, self.D)[:n], np.repeat(ok, self.T)[:n]

    def vmax(self):
        if self.fmt != "fp8":
            return 6 * 448 * float(self.gv)
        s = 1.0 if self.vs is None else float(self.vs)
        return 448 * s * (1.0 if self.vb is None else float(self.vb.max()))

    def check(self, got, only=None):
        out, lse = got
        G = self.G
        for b in range(len(self.lens)) if only is None else only:
            for h in range(self.H):
                rows = slice(h * G, (h + 1) * G)
                k, v, ok = self.tokens(b, h)
                n = self.lens[b]
                here = np.repeat(plain_windows.visible([n - 1], n, self.window, self.sinks) & ok, G, 0)
                plain_windows.check((out[b, rows], lse[b, rows]), self.q[b, rows].double().numpy(), k, v, here, self.sm, self.vmax(),
                                    blocks=self.fmt == "fp8")


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D,H,G", [(64, 2, 8), (128, 3, 4), (256, 2, 3), (128, 1, 1), (64, 5, 5)])
@pytest.mark.parametrize("T", [16, 48, 64, 128])
def test_windows(kv, cuda, fmt, D, H, G, T):
    """Windows and first tokens that end inside pages and tiles, over sequences shorter and longer than both."""
    for window, sinks in ((1, 0), (100, 4), (33, 70), (64, 64), (500, 1), (2000, 5)):
        c = Cache(cuda, fmt, [1, 0, 17, 64, 100, 101, 104, 128, 333, 1000, 1], H, T, D, G, window, sinks, seed=T + window)
        c.check(c.run(kv))


@pytest.mark.parametrize("D,H,G", [(64, 4, 6), (128, 8, 4), (256, 2, 8)])
@pytest.mark.parametrize("blocks", [True, False])
def test_fp8_without_a_window(kv, cuda, D, H, G, blocks):
    for T, lens in ((16, [1, 15, 16, 17, 31, 33, 0, 1000]), (64, [4000, 1, 64, 65, 0, 0, 129]), (112, [500, 113])):
        c = Cache(cuda, "fp8", lens, H, T, D, G, seed=T, blocks=blocks)
        c.check(c.run(kv))


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_sequences_are_cut_and_joined(kv, cuda, fmt, D):
    """One and two sequences over all SMs, many pieces a pair; a workspace of garbage."""
    for lens, window, sinks in (([40000], 0, 0), ([9000, 30011], 20000, 300), ([70001], 6000, 40)):
        if fmt == "nvfp4" and not window:
            window = 39000
        c = Cache(cuda, fmt, lens, 1, 64, D, 4, window, sinks, seed=len(lens))
        size = (kv.nvfp4_paged_fp8_decode_workspace_size if fmt == "fp8" else kv.nvfp4_paged_window_decode_workspace_size)
        ws = torch.randint(0, 256, (size(c.layout(kv), len(lens), 4, c.maxp),), dtype=torch.uint8, device=cuda)
        first = c.run(kv, workspace=ws)
        c.check(first)
        again = c.run(kv, workspace=ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_a_window_as_wide_as_the_sequences_is_the_dense_decode(kv, cuda):
    """Bit for bit: the same stages, runs and roundings."""
    c = Cache(cuda, "nvfp4", [3000, 64, 0, 999], 4, 64, 128, 4, window=3000, sinks=7, seed=3)
    out, lse = c.run(kv)
    d = lambda t: t.to(cuda)  # noqa: E731
    o2 = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device=cuda)
    l2 = torch.empty(c.q.shape[:2], device=cuda)
    kv.nvfp4_paged_decode_attention(c.layout(kv), d(c.q), d(c.kd), d(c.ksc), d(c.gk), d(c.vd), d(c.vsc), d(c.gv), d(c.table),
                                    torch.tensor(c.lens, dtype=torch.int32, device=cuda), c.sm, o2, lse=l2)
    assert np.array_equal(out, o2.double().cpu().numpy()) and np.array_equal(lse, l2.double().cpu().numpy())


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_pages_and_lengths(kv, cuda, fmt, D):
    """Ids outside the pool: their tokens are left out, all of them in one sequence. Lengths outside the table: nothing."""
    c = Cache(cuda, fmt, [200, 150, 64, 90], 2, 16, D, 2, window=120, sinks=20, seed=D)
    c.table[0, 12], c.table[0, 7], c.table[0, 0] = c.P, -1, 2 ** 31 - 1
    c.table[2, :] = -1
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = c.run(kv, status=status)
    c.check(got)
    assert status.item() == kv.STATUS_PAGE_OOB
    status.zero_()
    out, lse = c.run(kv, lens=[-1, c.maxp * 16 + 1, -2 ** 31, 2 ** 31 - 1], status=status)
    assert (out == 0).all() and (lse == -np.inf).all() and status.item() == kv.STATUS_BAD_SEQ_LEN


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_is_hidden_may_be_anything(kv, cuda, fmt, D):
    """NaN bytes in the tokens that the window hides, in those past the end and, for FP8, in the scales of pages without a
    visible token."""
    c = Cache(cuda, fmt, [70, 200, 37], 1, 32, D, 4, window=40, sinks=3, seed=5, drop=False)
    want = c.run(kv)
    for b, n in enumerate(c.lens):
        for j, page in enumerate(c.table[b].tolist()):
            if not 0 <= page < c.P:
                continue
            for t in range(32):
                at = j * 32 + t
                if at < n and (at >= n - 40 or at < 3):
                    continue
                if fmt == "fp8":
                    c.k[page, :, t], c.v[page, :, t] = 0x7F, 0xFF
                else:
                    c.ksc[page, :, t], c.vsc[page, :, t // 2, :, t % 2] = 0x7F, 0xFF
            if fmt == "fp8" and all(j * 32 + t >= n or (j * 32 + t < n - 40 and j * 32 + t >= 3) for t in range(32)):
                c.kb[page], c.vb[page] = float("nan"), float("inf")
    got = c.run(kv)
    assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])


def test_scales_of_pages_far_apart(kv, cuda):
    """V scales from 2^-40 to 2^30 within one sequence, scores that favour a page of a small one."""
    c = Cache(cuda, "fp8", [300, 64], 1, 16, 64, 4, seed=4)
    c.vb = 2.0 ** torch.randint(-40, 31, c.vb.shape, generator=c.g).float()
    c.kb = torch.full_like(c.kb, 0.01)
    small = c.table[0, 5]
    c.vb[small], c.kb[small] = 2.0 ** -38, 0.3
    got = c.run(kv)
    for b in range(2):
        k, v, ok = c.tokens(b, 0)
        q, here = c.q[b].double().numpy(), np.ones((4, c.lens[b]), bool)
        _, lse = plain_windows.attention(q, k, v, here, c.sm)
        # FP16 weights are subnormal against the largest product of weight and scale, not against the largest scale (a
        # token's largest E4M3 value among 64 is over 448 / 4)
        w = np.exp(q @ k.T * c.sm - lse[:, None])
        vmax = 4 * (w * np.abs(v).max(-1)).max(-1, keepdims=True)
        assert np.abs(plain_windows.FP8[c.v.numpy()[c.table[b, :c.lens[b] // 16].numpy(), 0]]).max(-1).min() >= 112
        plain_windows.check((got[0][b], got[1][b]), q, k, v, here, c.sm, vmax, blocks=True, logs=41)


def test_on_another_stream_and_captured(kv, cuda):
    """The two attentions captured into one graph on a side stream, replayed over new lengths and queries."""
    a = Cache(cuda, "fp8", [500, 1000, 3], 2, 64, 128, 4, window=300, sinks=10, seed=8, drop=False)
    b = Cache(cuda, "nvfp4", [500, 1000, 3], 2, 64, 128, 4, window=300, sinks=10, seed=9, drop=False)
    side = torch.cuda.Stream()
    lens = torch.tensor([1, 1, 1], dtype=torch.int32, device=cuda)
    outs = []
    pools, scales = a.fp8()
    d = lambda t: t.to(cuda)  # noqa: E731
    nv = [d(t) for t in (b.kd, b.ksc, b.gk, b.vd, b.vsc, b.gv)]
    q, ta, tb = d(a.q), d(a.table), d(b.table)
    oa, ob = torch.empty_like(q), torch.empty_like(q)
    wa = torch.empty(kv.nvfp4_paged_fp8_decode_workspace_size(a.layout(kv), 3, 8, a.maxp), dtype=torch.uint8, device=cuda)
    wb = torch.empty_like(wa)

    def step():
        kv.nvfp4_paged_fp8_decode_attention(a.layout(kv), q, *pools, ta, lens, a.sm, oa, window=300, sink_tokens=10, workspace=wa, **scales)
        kv.nvfp4_paged_window_decode_attention(b.layout(kv), q, *nv[:3], *nv[3:], tb, lens, b.sm, ob, window=300, sink_tokens=10, workspace=wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in ([500, 1000, 3], [320, 77, 0], [499, 311, 2]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for w in (wa, wb):
            w.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        outs = [oa.clone(), ob.clone()]
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        assert torch.equal(outs[0], oa) and torch.equal(outs[1], ob)
        a.lens = b.lens = n
        b.q = a.q
        for c, o in ((a, outs[0]), (b, outs[1])):
            k = c.run(kv)
            assert np.array_equal(k[0], o.double().cpu().numpy())
            c.check(k)
