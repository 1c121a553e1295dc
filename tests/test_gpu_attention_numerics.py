"""Both decode attentions against a 64-bit form with bounds that follow from what the kernels round, at scores of
every size and over pairs cut in every way.

With x a token's score in log2 units, p = 2^(x - m) and m near the largest x, the kernels round

  x    a sum of D exact products in FP32: at most 2^-23 of sum |products| for each of the D additions (nothing where
       every partial sum has 24 bits or fewer); the product with the scale, 2^-24 |x|; the scale itself, 3 2^-24 |x|,
       alike for all tokens of a head, so that it moves weights by their distance in x alone
  p    2^-22 (the approximate 2^y), then, before P V, to FP16: 2^-11, and 2^-25 where p is subnormal (against a largest p
       of at least 2^-1)
  sums FP32: 2^-23 of sum |terms| for each of n additions, 2^-21 for the join
  out  to BF16: half a step

so that |out - exact| <= half a step + A (2^-11 + 2 (2^-22 + dx + 2^-23 n) + 2^-21) + 2^-24 n max|v|, with
A = sum of weight |v| and dx = ln2 (2^-24 (2 max|x| + 3 (max x - min x)) + 2 2^-23 D S) what two scores may move
apart (S = largest sum of |products| of a token, in units of x). The factor 2: a weight's own error enters through
the sum of products and through the sum of the weights (2^-22, dx and n terms)."""
import numpy as np
import pytest
import torch

import plain_steps

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


class Pool:
    """An NVFP4 pool on the host and the GPU; codes and scales random, or set by a test before `to_device`."""

    def __init__(self, dev, P, H, T, D, seed, scale=(0x28, 0x39), sm=None, gk=0.8, gv=0.6):
        g = self.g = torch.Generator().manual_seed(seed)
        u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
        self.dev, self.P, self.H, self.T, self.D = dev, P, H, T, D
        self.kd, self.vd = u(0, 256, P, H, T, D // 2), u(0, 256, P, H, T // 2, D)
        self.ks, self.vs = u(*scale, P, H, T, D // 16), u(*scale, P, H, T // 2, D // 16, 2)
        self.sm = float(np.float32(D ** -0.5 if sm is None else sm))
        self.gk, self.gv = float(np.float32(gk)), float(np.float32(gv))

    def to_device(self):
        self.pool = [t.to(self.dev) for t in (self.kd, self.ks, self.vd, self.vs)]
        self.g_dev = [torch.tensor([x], device=self.dev) for x in (self.gk, self.gv)]
        return self

    def args(self, kv, q):
        kd, ks, vd, vs = self.pool
        return kv.Layout(self.H, self.D, self.T), q.to(self.dev), kd, ks, self.g_dev[0], vd, vs, self.g_dev[1]

    def outputs(self, q):
        return (torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=self.dev),
                torch.full(q.shape[:2], float("nan"), device=self.dev))

    def sparse(self, kv, q, table, lens, **kw):
        out, lse = self.outputs(q)
        kv.nvfp4_paged_sparse_decode_attention(*self.args(kv, q), table.to(self.dev), lens.to(self.dev), self.sm, out,
                                               lse=lse, **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def dense(self, kv, q, table, lens, **kw):
        out, lse = self.outputs(q)
        kv.nvfp4_paged_decode_attention(*self.args(kv, q), table.to(self.dev), lens.to(self.dev), self.sm, out, lse=lse,
                                        **kw)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, got, q, table, lens, exact_sums=False, run=None, records=0):
        """table [B, H, pages], lens [B, H]: every row of `got` within the bound at the top of this file, S left out
        where the sums of products are exact. Pairs known to be cut into runs of at most `run` tokens, joined from
        `records` of them, sum that many terms each (and a run's weights are held against a maximum of its own)."""
        out, lse = got
        B, Hq, D = q.shape
        G, T = Hq // self.H, self.T
        kd, ks, vd, vs = (t.numpy() for t in (self.kd, self.ks, self.vd, self.vs))
        qd = q.double().numpy()
        assert np.isfinite(out).all()
        scale = self.sm * self.gk
        for b in range(B):
            for h in range(self.H):
                n, rows = int(lens[b, h]), slice(h * G, (h + 1) * G)
                if n == 0:
                    assert (out[b, rows] == 0).all() and (lse[b, rows] == -np.inf).all()
                    continue
                ids = table[b, h, :-(-n // T)].numpy()
                k = plain_steps.keys(kd[ids, h], ks[ids, h]).reshape(-1, D)[:n]
                code = np.stack([vd[ids, h] & 15, vd[ids, h] >> 4], 2)
                v = plain_steps.E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
                sc = plain_steps.E4M3[np.moveaxis(vs[ids, h], -1, -2)]
                v = (v.reshape(*v.shape[:-1], -1, 16) * sc[..., None]).reshape(-1, D)[:n]
                x = qd[b, rows] @ k.T * scale
                top = x.max(-1, keepdims=True)
                p = np.exp(x - top)
                want_lse = (top + np.log(p.sum(-1, keepdims=True)))[:, 0]
                w = np.exp(x - want_lse[:, None])
                want, A = w @ v * self.gv, w @ np.abs(v) * self.gv
                S = 0.0 if exact_sums else (np.abs(qd[b, rows]) @ np.abs(k).T).max(-1) * abs(scale) * LOG2E
                big = np.abs(x).max(-1) * LOG2E
                dist = (top[:, 0] - x.min(-1)) * LOG2E
                dx = (np.log(2) * (2.0 ** -24 * (2 * big + 3 * dist) + 2 * 2.0 ** -23 * D * S))[:, None]
                terms = n if run is None else min(n, run) + records
                rel = 2.0 ** -11 + 2 * (2.0 ** -22 + dx + 2.0 ** -23 * terms) + 2.0 ** -21
                tol = A * rel + 2.0 ** -24 * (n if run is None else min(n, run)) * np.abs(v).max() * self.gv
                half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want) + tol, 2.0 ** -126))) - 8)
                err = np.abs(out[b, rows] - want)
                assert (err <= tol + half).all(), (b, h, n, float((err - tol - half).max()))
                # the scale's three roundings, x's own, that of m + log2(l), and two of its product with ln 2
                ltol = 2.0 ** -24 * (3 + 1 + 3) * np.maximum(big, np.abs(want_lse) * LOG2E) + dx[:, 0] + 2.0 ** -22 * terms + 2.0 ** -20
                assert (np.abs(lse[b, rows] - want_lse) <= ltol).all(), (b, h, n, lse[b, rows] - want_lse, ltol)


# ------------------------------------------------------------------------------------ scores of every size

def parts(x):
    """x (a multiple of 4) as a sum of 4 times three BF16 integers."""
    out, left = [], x // 4
    for _ in range(3):
        shift = max(0, abs(left).bit_length() - 8)
        hi = (abs(left) >> shift << shift) * (1 if left >= 0 else -1)
        out.append(hi)
        left -= hi
    assert left == 0
    return out


def keys_of_one_score(c, spread):
    """All keys alike in dims 0 .. 2 (4.0 each); with `spread` they differ by up to 48 in dims 16 .. 31."""
    c.kd[:], c.ks[:] = 0, 0x38   # scale 1
    c.kd[..., 0], c.kd[..., 1] = 0x66, 0x06
    if spread:
        c.kd[..., 8:16] = torch.randint(0, 256, c.kd[..., 8:16].shape, generator=c.g, dtype=torch.uint8)


def queries_of_scores(c, B, G, scores):
    """Head g of every pair scores scores[g % len] log2 units over the common dims."""
    q = torch.zeros((B, c.H, G, c.D))
    q[..., 16:32] = 1.0
    for g in range(G):
        q[:, :, g, :3] = torch.tensor(parts(scores[g % len(scores)]), dtype=torch.float32)
    q = q.reshape(B, c.H * G, c.D)
    assert torch.equal(q, q.to(torch.bfloat16).float())
    return q.to(torch.bfloat16)


# Around the bound of the FP16 maximum (4096), where its steps are 16 and 32 (a maximum rounded half a step too
# low), around its largest value (65504), and far past it.
SIZES = [0, 2044, 4092, 4100, 21512, 32784, 45400, 65472, 65520, 70000, 144000, 1000000]


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_every_size_and_sign(kv, cuda, D, size, spread):
    """One token, part of a stage, one stage, one token more, and pairs split over several warps; heads of one pair
    at +size, -size and 0 beside one another, and all at -size."""
    T, H, most = 16, 2, 44
    c = Pool(cuda, 12, H, T, D, D + size, sm=np.log(2.0), gk=1.0, gv=1.0)
    keys_of_one_score(c, spread)
    c.to_device()
    lens = torch.tensor([[1, 63], [64, 65], [most * T, 0], [17, 333]], dtype=torch.int32)
    B = lens.shape[0]
    table = torch.randint(0, 12, (B, H, most), generator=c.g, dtype=torch.int32)
    same, one = table[:, :1].expand(B, H, most).contiguous(), lens[:, :1].expand(B, H).contiguous()
    for scores in ([size, -size, 0, -size], [-size]):
        q = queries_of_scores(c, B, 4, scores)
        c.check(c.sparse(kv, q, table, lens), q, table, lens, True)
        c.check(c.dense(kv, q, same[:, 0].contiguous(), one[:, 0].contiguous()), q, same, one, True)
        for splits in (1, 5):
            c.check(c.dense(kv, q, same[:, 0].contiguous(), one[:, 0].contiguous(), max_num_splits=splits), q, same, one,
                    True)


@pytest.mark.parametrize("size", [45400, 70000])
def test_negative_scores_over_many_pairs(kv, cuda, size):
    """1200 pairs in runs that cross pairs (records joined through global memory), every score far below zero."""
    T, H, D, B, most = 16, 4, 128, 300, 9
    c = Pool(cuda, 20, H, T, D, size, sm=np.log(2.0), gk=1.0, gv=1.0)
    keys_of_one_score(c, True)
    c.to_device()
    lens = torch.randint(0, most * T + 1, (B, H), generator=c.g, dtype=torch.int32)
    table = torch.randint(0, 20, (B, H, most), generator=c.g, dtype=torch.int32)
    q = queries_of_scores(c, B, 2, [-size, 0])
    c.check(c.sparse(kv, q, table, lens), q, table, lens, True)


# ------------------------------------------------------------------------------------ pairs of every length and cut

def touched(kv, c, q, table, lens, **kw):
    """The outputs over a workspace of garbage, twice the same, and the bytes of it that the call wrote (0 where each
    pair was cut within a cluster of CTAs)."""
    B, Hq, D = q.shape
    n = kv.nvfp4_paged_sparse_decode_workspace_size(kv.Layout(c.H, D, c.T), B, Hq, table.shape[2])
    w = torch.full((n,), 0xA5, dtype=torch.uint8, device=c.dev)
    got = c.sparse(kv, q, table, lens, workspace=w, **kw)
    again = c.sparse(kv, q, table, lens, workspace=w, **kw)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])
    return got, int((w != 0xA5).sum())


@pytest.mark.parametrize("B,H,G,D,T,pages,own", [
    (1, 8, 4, 128, 64, 64, True), (2, 4, 8, 256, 16, 70, True), (1, 5, 1, 64, 32, 128, True),  # clusters of 8 CTAs
    (8, 4, 8, 64, 64, 40, True), (8, 8, 2, 128, 64, 30, True),                                 # of 4 and 2
    (19, 8, 4, 128, 64, 32, True), (75, 4, 2, 128, 64, 20, True),                              # one CTA a pair, and two
    (20, 8, 1, 64, 64, 64, False), (19, 5, 3, 256, 16, 150, False), (40, 8, 4, 128, 64, 32, False),  # over all pairs
])
def test_long_pairs_within_the_bound_of_their_roundings(kv, cuda, B, H, G, D, T, pages, own):
    """Averages of about 1000 to 4000 tokens, outputs of a few hundredths, against the derived bound (about
    2^-10 of the mean |v|), cut within clusters (`own`: the workspace is left alone) or into runs over all pairs; the
    dense kernel over the same pages."""
    c = Pool(cuda, 60, H, T, D, B + pages).to_device()
    lens = torch.randint(pages * T // 2, pages * T + 1, (B, H), generator=c.g, dtype=torch.int32)
    table = torch.randint(0, 60, (B, H, pages), generator=c.g, dtype=torch.int32)
    q = torch.randn((B, H * G, D), generator=c.g).to(torch.bfloat16)
    got, wrote = touched(kv, c, q, table, lens)
    assert (wrote == 0) == own
    c.check(got, q, table, lens)
    same, one = table[:, :1].expand(B, H, pages).contiguous(), lens[:, :1].expand(B, H).contiguous()
    c.check(c.dense(kv, q, same[:, 0].contiguous(), one[:, 0].contiguous()), q, same, one)


@pytest.mark.parametrize("D,G,T,n", [(128, 1, 128, 38400), (256, 3, 128, 50000), (64, 2, 64, 100000), (128, 8, 128, 150000),
                                      (256, 1, 16, 30000)])
def test_a_pair_of_more_records_than_shared_memory_holds(kv, cuda, D, G, T, n):
    """One long pair beside a short and an empty one, cut into 600 to 1600 runs: their records are joined in chunks.
    What the call writes of the workspace shows the records: G (D + 2) floats each."""
    pages = -(-n // T)
    c = Pool(cuda, 50, 1, T, D, n).to_device()
    lens = torch.tensor([[n], [70], [0]], dtype=torch.int32)
    table = torch.randint(0, 50, (3, 1, pages), generator=c.g, dtype=torch.int32)
    q = torch.randn((3, G, D), generator=c.g).to(torch.bfloat16)
    got, wrote = touched(kv, c, q, table, lens)
    record = G * (D + 2) * 4
    held = 227 * 1024 // record
    assert wrote > 0.9 * record * (held + 1), (wrote, record)
    # 1600 runs and more (8 warps an SM and up): at most 3 stages each
    c.check(got, q, table, lens, run=4 * 64, records=2500)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_token_pairs_return_their_value_rows(kv, cuda, D):
    """A single token's output is its V row, rounded to FP16 against its own weight and to BF16, whatever its score."""
    B, H, G, T = 64, 4, 3, 16
    c = Pool(cuda, 40, H, T, D, D, scale=(0x20, 0x50)).to_device()
    lens = torch.ones((B, H), dtype=torch.int32)
    table = torch.randint(0, 40, (B, H, 2), generator=c.g, dtype=torch.int32)
    q = (torch.randn((B, H * G, D), generator=c.g) * 10.0 ** torch.randint(-3, 3, (B, H * G, 1), generator=c.g)).to(torch.bfloat16)
    c.check(c.sparse(kv, q, table, lens), q, table, lens)
