"""FP8 pages of runs with NaN and infinities: one rule for runs of all sizes and sources."""
import numpy as np
import pytest
import torch

from test_gpu_extend_attention import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def encode(kv, lay, src, tokens=None, **kw):
    P, H, T, D = src.shape[0], lay.num_kv_heads, lay.page_size, lay.head_dim
    dst, scales = torch.full((P, H, T, D), 0x55, dtype=torch.uint8, device=src.device), torch.full((P, H), -5.0, device=src.device)
    tokens = None if tokens is None else torch.tensor(tokens, dtype=torch.int32, device=src.device)
    kv.nvfp4_kv_fp8_pages(lay, src, dst, scales, page_tokens=tokens, **kw)
    return dst.cpu(), scales.cpu()


SHAPES = [(16, 128), (64, 128), (1, 16), (16, 64), (130, 256), (512, 256), (6, 80)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sign", [1, -1])
def test_16_bit(kv, cuda, T, D, dtype, sign):
    """One NaN or infinity at the run's begin, in the middle, at its last valid token; the other head as without it."""
    H, m = 2, T - T // 4
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn((3, H, T, D), generator=g).to(dtype).to(cuda)
    lay = kv.Layout(H, D, T)
    clean, scales = encode(kv, lay, x, [m] * 3)
    for value in (float("nan"), float("inf")):
        y = x.clone()
        for page, (t, d) in enumerate(((0, 0), (m // 2, D - 1), (m - 1, D // 2))):
            y[page, 1, t, d] = sign * value
        got, s = encode(kv, lay, y, [m] * 3)
        assert torch.equal(got[:, 0], clean[:, 0]) and torch.equal(s[:, 0], scales[:, 0])
        want = torch.zeros((3, T, D), dtype=torch.uint8)
        if value != value:
            want[:, :m] = 0x7F
            assert bool(s[:, 1].isnan().all())
        else:
            for page, (t, d) in enumerate(((0, 0), (m // 2, D - 1), (m - 1, D // 2))):
                want[page, t, d] = 0x7F
            got[:, 1] = torch.where((got[:, 1] & 0x7F) != 0, got[:, 1] & 0x7F, 0)   # (signs of zeros and of NaN aside)
            assert bool(s[:, 1].isinf().all())
        assert torch.equal(got[:, 1], want)


@pytest.mark.parametrize("T,D", [s for s in SHAPES if s[0] % 2 == 0])
@pytest.mark.parametrize("pairs", [False, True])
def test_nvfp4(kv, cuda, T, D, pairs):
    """A NaN among the block scales, and a NaN global scale."""
    H, m = 2, T - T // 4
    g = torch.Generator().manual_seed(T + D)
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8).to(cuda)  # noqa: E731
    data = u(0, 256, 2, H, T // 2, D) if pairs else u(0, 256, 2, H, T, D // 2)
    sc = u(0x28, 0x39, 2, H, T // 2, D // 16, 2) if pairs else u(0x28, 0x39, 2, H, T, D // 16)
    lay = kv.Layout(H, D, T, kv.PACK_TOKEN_PAIRS if pairs else kv.PACK_DIM_PAIRS)
    one = torch.tensor([0.5], device=cuda)
    clean, scales = encode(kv, lay, data, [m] * 2, src_scales=sc, global_scale=one)
    bad = sc.clone()
    for page, t in ((0, 0), (1, m - 1)):
        if pairs:
            bad[page, 1, t // 2, -1, t % 2] = 0x7F
        else:
            bad[page, 1, t, 0] = 0x7F
    got, s = encode(kv, lay, data, [m] * 2, src_scales=bad, global_scale=one)
    assert torch.equal(got[:, 0], clean[:, 0]) and torch.equal(s[:, 0], scales[:, 0]) and bool(s[:, 1].isnan().all())
    assert bool((got[:, 1, :m] == 0x7F).all()) and not bool(got[:, 1, m:].any())
    got, s = encode(kv, lay, data, [m] * 2, src_scales=sc, global_scale=one * float("nan"))
    assert bool(s.isnan().all()) and bool((got[:, :, :m] == 0x7F).all()) and not bool(got[:, :, m:].any())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_chunk_with_one_bad_token(kv, cuda, value):
    """Encoded and attended to: rows before the token's page are as without it, rows that see it are NaN."""
    c = Chunk(cuda, [300], [200], 1, 16, 128, 4, seed=1)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((c.P, 1, 16, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    c.ks = c.vs = None

    def attend(k, v):
        (c.k, c.kb), (c.v, c.vb) = (encode(kv, c.layout(kv), x.to(cuda)) for x in (k, v))
        return c.run(kv)
    want = attend(k, v)
    at = 250  # of page 15: tokens 240 .. 255
    for x in (k, v):
        y = x.clone()
        y[c.table[0, at // 16], 0, at % 16, 5] = value
        got = attend(y if x is k else k, y if x is v else v)
        for a, b in zip(got, want):
            assert (a[:240 - 100] == b[:240 - 100]).all()
        assert np.isnan(got[0][at - 100:]).any(-1).all()
