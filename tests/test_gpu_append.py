"""GPU append of rows to the NVFP4 cache against its plain 64-bit form. Codes, scales and the 16-bit
outputs are exact: every FP32 rounding of the rotation and of the encoder is part of the definition,
and q_out, k_out, v_out round one FP32 value to nearest even, so there is no tolerance."""
import numpy as np
import pytest
import torch

import plain_steps

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def random_pool(P, H, T, D, g):
    b = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    return {"kd": b(P, H, T, D // 2), "ks": b(P, H, T, D // 16), "vd": b(P, H, T // 2, D), "vs": b(P, H, T // 2, D // 16, 2)}


def table_of(n, dims, base=10000.0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Case:
    """Inputs on the host and on the GPU, the q, k, v slices of one projection."""

    def __init__(self, dev, rows, Hq, H, D, T, P, slots, dtype="bf16", seed=0, far=5000, wide=True, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.D, self.T, self.Hq, self.dev = H, D, T, Hq, dev
        pad = 0 if wide else 8
        w = (Hq + 2 * H) * D + pad
        x = torch.randn((rows, w), generator=g) * spread
        x[:, Hq * D:Hq * D + D:16] *= 20
        x = x.to(DT[dtype])
        self.base = x.to(dev)
        cut = lambda t: (t[:, :Hq * D].view(rows, Hq, D), t[:, Hq * D:(Hq + H) * D].view(rows, H, D),  # noqa: E731
                         t[:, (Hq + H) * D:(Hq + 2 * H) * D].view(rows, H, D))
        self.q, self.k, self.v = cut(self.base)
        self.hq, self.hk, self.hv = (t.double().numpy() for t in cut(x))
        self.slots = torch.as_tensor(slots, dtype=torch.int64)
        self.positions = torch.randint(0, far, (rows,), generator=g, dtype=torch.int32)
        self.pool = random_pool(P, H, T, D, g)
        self.gk, self.gv = np.float32(0.013), np.float32(0.0021)

    def run(self, kv, rot=None, outs=torch.bfloat16, status=None, with_q=True, pool=None, stream=None):
        dev, rows = self.dev, len(self.slots)
        pool = {k: v.to(dev) for k, v in self.pool.items()} if pool is None else pool
        o = [torch.full((rows, h, self.D), 7.0, dtype=outs, device=dev) for h in (self.Hq, self.H, self.H)]
        kw = {}
        if with_q and self.Hq:
            kw.update(q=self.q, q_out=o[0])
        if rot is not None:
            style, first, dims, table = rot
            kw.update(rotary=kv.Rotary(kv.ROTARY_HALVES if style == "halves" else kv.ROTARY_PAIRS, first, dims,
                                       table.to(dev)), positions=self.positions.to(dev))
        kv.nvfp4_kv_append(kv.Layout(self.H, self.D, self.T), self.k, self.v, self.slots.to(dev), pool["kd"], pool["ks"],
                           pool["vd"], pool["vs"], k_out=o[1], v_out=o[2],
                           k_global_scale=torch.tensor([self.gk], device=dev),
                           v_global_scale=torch.tensor([self.gv], device=dev), status=status, stream=stream, **kw)
        torch.cuda.synchronize()
        return {k: v.cpu().numpy() for k, v in pool.items()}, [t.cpu() for t in o]

    def want(self, rot=None):
        pool = {k: v.clone().numpy() for k, v in self.pool.items()}
        r = None if rot is None else (*rot[:3], rot[3].numpy())
        return pool, plain_steps.append(pool, self.hk, self.hv, self.slots.numpy(), self.T, self.gk, self.gv, r,
                                        self.positions.numpy(), self.hq)

    def check(self, got, want, outs=torch.bfloat16, with_q=True):
        (pool, o), (wpool, wo) = got, want
        for name in ("ks", "kd", "vs", "vd"):
            assert np.array_equal(pool[name], wpool[name]), name
        for t, rows, skip in zip(o, wo, (not with_q, False, False)):
            for n, w in enumerate(rows):
                if w is None or skip:
                    assert (t[n] == 7.0).all(), n
                else:
                    assert torch.equal(t[n], torch.from_numpy(w).float().to(outs)), n


def some_slots(kind, rows, P, T, seed):
    rng = np.random.default_rng(seed)
    if kind == "run":                      # one sequence, from an odd slot on
        return np.arange(rows) + 1
    if kind == "shuffled":                 # partners far apart in the call, or missing
        return rng.permutation(P * T)[:rows]
    if kind == "backwards":                # second tokens before first ones
        return np.arange(rows)[::-1].copy() + T - 1
    s = rng.permutation(P * T)[:rows]      # padding rows among the others
    s[rng.random(rows) < 0.4] = -1
    s[0] = -1
    return s


@pytest.mark.parametrize("kind", ["run", "shuffled", "backwards", "padded"])
@pytest.mark.parametrize("D,T,Hq,H,dtype,style,first,dims", [
    (128, 64, 8, 2, "bf16", "halves", 0, 128), (64, 16, 3, 3, "fp16", "pairs", 0, 64),
    (256, 32, 5, 1, "bf16", "pairs", 192, 64), (128, 2, 7, 7, "fp16", "halves", 16, 96),
    (256, 48, 4, 2, "fp16", "halves", 48, 128), (64, 6, 9, 1, "bf16", "halves", 16, 32)])
def test_rows_of_every_kind(kv, cuda, kind, D, T, Hq, H, dtype, style, first, dims):
    P = 200 // T + 2
    c = Case(cuda, 37, Hq, H, D, T, P, some_slots(kind, 37, P, T, D + T), dtype, seed=T, wide=T != 16)
    rot = (style, first, dims, table_of(5000, dims))
    outs = torch.float16 if T == 48 else torch.bfloat16
    c.check(c.run(kv, rot, outs), c.want(rot), outs)


@pytest.mark.parametrize("rows", [1, 2, 3, 700])
def test_numbers_of_rows_without_rotation(kv, cuda, rows):
    """700 rows of 12 + 2 x 6 heads: more head groups than the warps that one head group each would
    fill, so a warp takes whole rows."""
    P, T = rows // 32 + 2, 32
    c = Case(cuda, rows, 48 if rows == 700 else 6, 6, 128, T, P, np.arange(rows) + 5, seed=rows)
    c.check(c.run(kv), c.want())
    c.check(c.run(kv, with_q=False), c.want(), with_q=False)


def test_whole_rows_per_warp_with_rotation(kv, cuda):
    """Head groups above 32 per SM (a warp then loops over the head groups of a row)."""
    rows, T, P = 1300, 64, 24
    c = Case(cuda, rows, 24, 3, 64, T, P, some_slots("padded", rows, P, T, 1), "bf16", seed=9)
    rot = ("pairs", 0, 32, table_of(5000, 32))
    c.check(c.run(kv, rot), c.want(rot))


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 3e3, 1e4])
def test_small_and_large_values(kv, cuda, spread):
    """Block scales that round to zero or saturate."""
    c = Case(cuda, 9, 4, 2, 64, 16, 3, np.arange(9) * 2, "bf16", seed=3, spread=spread)
    rot = ("halves", 0, 64, table_of(5000, 64))
    c.check(c.run(kv, rot), c.want(rot))


def test_equals_the_page_quantizer(kv, cuda):
    """Whole pages appended a token at a time are the page quantizer's bytes."""
    P, H, T, D = 5, 3, 32, 128
    g = torch.Generator().manual_seed(4)
    pages = {n: torch.randn((P, H, T, D), generator=g).to(torch.bfloat16).to(cuda) for n in "kv"}
    gs = torch.tensor([0.002], device=cuda)
    lay = kv.Layout(H, D, T)
    e = lambda *s: torch.zeros(s, dtype=torch.uint8, device=cuda)  # noqa: E731
    a = [e(P, H, T, D // 2), e(P, H, T, D // 16), e(P, H, T, D // 2), e(P, H, T, D // 16)]
    b = [torch.zeros_like(t) for t in a]
    kv.nvfp4_kv_quantize_pages(lay, pages["k"], gs, a[0], a[1])
    kv.nvfp4_kv_quantize_pages(lay.with_packing(kv.PACK_TOKEN_PAIRS), pages["v"], gs, a[2], a[3])
    order = torch.randperm(P * T, generator=g)
    rows = {n: t.transpose(1, 2).reshape(P * T, H, D)[order.to(cuda)].contiguous() for n, t in pages.items()}
    k_out, v_out = torch.empty_like(rows["k"]), torch.empty_like(rows["v"])
    kv.nvfp4_kv_append(lay, rows["k"], rows["v"], order.to(cuda), *b, k_global_scale=gs, v_global_scale=gs,
                       k_out=k_out, v_out=v_out)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    back = torch.empty_like(pages["k"])
    for data, sc, out, pack in ((a[0], a[1], k_out, kv.PACK_DIM_PAIRS), (a[2], a[3], v_out, kv.PACK_TOKEN_PAIRS)):
        kv.nvfp4_kv_dequantize_pages(lay.with_packing(pack), data, sc, gs, back)
        assert torch.equal(back.transpose(1, 2).reshape(P * T, H, D)[order.to(cuda)], out)


def test_bad_slots_and_positions_skip_their_rows(kv, cuda):
    T, P = 16, 3
    c = Case(cuda, 8, 4, 2, 64, T, P, [0, 1, P * T, 3, -2, 5, 2 ** 40, 6], seed=5)
    rot = ("halves", 0, 64, table_of(100, 64))
    c.positions = torch.tensor([0, 100, 5, -1, 7, 99, 3, 2 ** 31 - 1], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    c.check(c.run(kv, rot, status=status), c.want(rot))
    assert status.item() == kv.STATUS_PAGE_OOB | kv.STATUS_BAD_POSITION
    c.positions[:] = 1
    c.slots = torch.tensor([4, 5, 9, 8, -1, 12, 13, 30])
    status.zero_()
    c.check(c.run(kv, rot, status=status), c.want(rot))
    assert status.item() == 0


def test_the_two_tokens_of_a_pair_from_two_streams(kv, cuda):
    """Even tokens on one stream, odd ones on another, at once: every V byte keeps both nibbles."""
    rows, T = 512, 64
    one = Case(cuda, rows, 0, 4, 128, T, 20, np.arange(rows) * 2, seed=6)
    two = Case(cuda, rows, 0, 4, 128, T, 20, np.arange(rows) * 2 + 1, seed=7)
    for rep in range(5):
        pool = {k: v.to(cuda) for k, v in one.pool.items()}
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for c, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                kv.nvfp4_kv_append(kv.Layout(4, 128, T), c.k, c.v, c.slots.to(cuda), pool["kd"], pool["ks"], pool["vd"],
                                   pool["vs"])
        torch.cuda.synchronize()
        want = {k: v.clone().numpy() for k, v in one.pool.items()}
        for c in (one, two):
            plain_steps.append(want, c.hk, c.hv, c.slots.numpy(), T, 1.0, 1.0)
        for n in want:
            assert np.array_equal(pool[n].cpu().numpy(), want[n]), n


def test_captured_and_replayed_with_new_rows(kv, cuda):
    """A decode step in a CUDA graph: rows, slots and positions change between replays."""
    T, P, rows = 16, 8, 6
    c = Case(cuda, rows, 4, 2, 64, T, P, np.arange(rows), seed=8)
    rot = ("halves", 0, 64, table_of(5000, 64))
    pool = {k: v.to(cuda) for k, v in c.pool.items()}
    slots, positions = c.slots.to(cuda), c.positions.to(cuda)
    r = kv.Rotary(kv.ROTARY_HALVES, 0, 64, rot[3].to(cuda))
    q_out = torch.zeros((rows, 4, 64), dtype=torch.bfloat16, device=cuda)
    gk, gv = torch.tensor([c.gk], device=cuda), torch.tensor([c.gv], device=cuda)

    def step():
        kv.nvfp4_kv_append(kv.Layout(2, 64, T), c.k, c.v, slots, pool["kd"], pool["ks"], pool["vd"], pool["vs"], q=c.q,
                           q_out=q_out, rotary=r, positions=positions, k_global_scale=gk, v_global_scale=gv)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = {k: v.clone().numpy() for k, v in c.pool.items()}
    plain_steps.append(want, c.hk, c.hv, c.slots.numpy(), T, c.gk, c.gv, (*rot[:3], rot[3].numpy()), c.positions.numpy())
    for i in range(1, 5):
        new = torch.tensor([(i * 7 + 13 * j) % (P * T) if j != i else -1 for j in range(rows)])
        slots.copy_(new)
        positions.copy_(positions.flip(0))
        c.base.copy_(torch.roll(c.base, 1, 0))
        graph.replay()
        torch.cuda.synchronize()
        hk, hv = c.k.double().cpu().numpy(), c.v.double().cpu().numpy()
        plain_steps.append(want, hk, hv, new.numpy(), T, c.gk, c.gv, (*rot[:3], rot[3].numpy()), positions.cpu().numpy())
        for n in want:
            assert np.array_equal(pool[n].cpu().numpy(), want[n]), n


def test_slots_past_32_bit_byte_offsets(kv, cuda):
    """A cache whose code pools pass 2^32 bytes: the first and the last page, and one past 2^32."""
    H, D, T = 8, 256, 128
    P = (1 << 32) // (H * T * D // 2) + 40
    pool = [torch.zeros(s, dtype=torch.uint8, device=cuda)
            for s in ((P, H, T, D // 2), (P, H, T, D // 16), (P, H, T // 2, D), (P, H, T // 2, D // 16, 2))]
    pages = [0, P - 40, P - 1]
    slots = torch.tensor([pages[0] * T, pages[1] * T + 6, pages[1] * T + 7, P * T - 1])
    c = Case(cuda, 4, 8, H, D, T, 1, slots, seed=11)
    kv.nvfp4_kv_append(kv.Layout(H, D, T), c.k, c.v, slots.to(cuda), *pool)
    small = {n: np.zeros((3, *t.shape[1:]), np.uint8) for n, t in zip(("kd", "ks", "vd", "vs"), pool)}
    plain_steps.append(small, c.hk, c.hv, [0, T + 6, T + 7, 3 * T - 1], T, 1.0, 1.0)
    for n, t in zip(("kd", "ks", "vd", "vs"), pool):
        assert np.array_equal(t[pages].cpu().numpy(), small[n]), n
        assert int(t[pages[0] + 1].sum()) == 0 and int(t[pages[1] + 1].sum()) == 0


def test_binding_refuses_on_the_gpu(kv, cuda):
    c = Case(cuda, 4, 4, 2, 64, 16, 3, np.arange(4))
    pool = [c.pool[n].to(cuda) for n in ("kd", "ks", "vd", "vs")]
    lay, slots = kv.Layout(2, 64, 16), c.slots.to(cuda)
    with pytest.raises(ValueError, match="contiguous"):
        kv.nvfp4_kv_append(lay, c.k.transpose(1, 2).contiguous().transpose(1, 2), c.v, slots, *pool)
    with pytest.raises(ValueError, match="q_out"):
        kv.nvfp4_kv_append(lay, c.k, c.v, slots, *pool, q=c.q)
    with pytest.raises(TypeError):
        kv.nvfp4_kv_append(lay, c.k, c.v.half(), slots, *pool)
    with pytest.raises(kv.NVFP4KVError, match="INVALID"):   # in place
        kv.nvfp4_kv_append(lay, c.k, c.v, slots, *pool, q=c.q, q_out=c.q)
    with pytest.raises(ValueError, match="positions"):
        kv.nvfp4_kv_append(lay, c.k, c.v, slots, *pool,
                           rotary=kv.Rotary(kv.ROTARY_HALVES, 0, 64, table_of(9, 64).to(cuda)))
    for bad in ((pool[0], pool[1], pool[2][:2], pool[3][:2]), (pool[0], pool[1][..., :1], pool[2], pool[3]),
                (pool[0].to(torch.int8), pool[1], pool[2], pool[3]), (pool[0].cpu(), *pool[1:])):
        with pytest.raises(ValueError):
            kv.nvfp4_kv_append(lay, c.k, c.v, slots, *bad)
    for bad in (slots[:3], slots.int(), slots.cpu(), slots.repeat(2)[::2]):
        with pytest.raises(ValueError, match="slots"):
            kv.nvfp4_kv_append(lay, c.k, c.v, bad, *pool)
