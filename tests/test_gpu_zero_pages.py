"""Attention over FP8 pages some of which hold no value at all: nvfp4_kv_fp8_pages gives them a scale of 1 beside the others'
small ones, and they count in the softmax alone."""
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


def encode(c, kv, amax, zero, ends=True):
    """The cache's pages encoded from 16-bit ones: V of `amax` and of 0 in the pages zero(b, j), whose keys are larger than the others';
    each with its valid tokens. -> the values [P, H, T, D] of V as encoded."""
    g, dev = c.g, c.dev
    shape = (c.P, c.H, c.T, c.D)
    k = torch.randn(shape, generator=g)
    v = torch.randn(shape, generator=g).clamp(-4, 4) * (amax / 4)
    tokens = torch.full((c.P,), c.T, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        for j in range(-(-n // c.T)):
            page = int(c.table[b, j])
            if not 0 <= page < c.P:
                continue
            if ends:
                tokens[page] = min(c.T, n - j * c.T)
            if zero(b, j):
                v[page], k[page] = 0.0, k[page] * 2.0
    k8, v8 = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2))
    kb, vb = (torch.zeros(shape[:2], device=dev) for _ in range(2))
    for x, x8, xb in ((k, k8, kb), (v, v8, vb)):
        kv.nvfp4_kv_fp8_pages(c.layout(kv), x.to(torch.bfloat16).to(dev), x8, xb, page_tokens=tokens.to(dev))
    c.k, c.v, c.kb, c.vb, c.ks, c.vs = k8.cpu(), v8.cpu(), kb.cpu(), vb.cpu(), None, None
    empty = [int(c.table[b, j]) for b, n in enumerate(c.lens) for j in range(-(-n // c.T)) if zero(b, j)]
    assert bool((c.vb[[e for e in empty if 0 <= e < c.P]] == 1).all())


def check(c, got, rows_of):
    """Rows of every sequence against 64 bits, with the largest |v| that its tokens have."""
    out, lse = got
    for b, n in enumerate(c.lens):
        rows, pos = rows_of(b, n)
        if n == 0 or len(pos) == 0:
            continue
        for h in range(c.H):
            k, v, ok = c.tokens(b, h)
            here = np.repeat(plain_windows.visible(pos, n, c.window, c.sinks) & ok, c.G, 0)
            heads = slice(h * c.G, (h + 1) * c.G)
            vmax = np.abs(v[here.any(0)]).max()
            plain_windows.check((out[rows, heads].reshape(-1, c.D), lse[rows, heads].reshape(-1)),
                                c.q[rows, heads].double().numpy().reshape(-1, c.D), k, v, here, c.sm, vmax, blocks=True, logs=60)


PATTERNS = {"first": lambda b, j: j == 0, "some": lambda b, j: j % 5 == 2, "most": lambda b, j: j % 4 != 1, "last": lambda b, j: j >= 5}


@pytest.mark.parametrize("amax", [1.0, 1e-3, 1e-5, 1e-9])
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("D,T", [(64, 16), (64, 64), (128, 16), (128, 48), (128, 64), (256, 16), (256, 64)])
def test_decode(kv, cuda, D, T, pattern, amax):
    for window, sinks in ((0, 0), (200, 20)):
        c = Cache(cuda, "fp8", [5 * T + 7, 700, 33, 0, 16 * T], 2, T, D, 4, window, sinks, seed=T + D)
        encode(c, kv, amax, PATTERNS[pattern])
        check(c, c.run(kv), lambda b, n: ([b], [n - 1]))


@pytest.mark.parametrize("amax", [1.0, 1e-3, 1e-5, 1e-9])
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("D,T", [(64, 16), (64, 64), (128, 16), (128, 48), (128, 64), (256, 16), (256, 64)])
def test_extend(kv, cuda, D, T, pattern, amax):
    for window, sinks in ((0, 0), (90, 20)):
        c = Chunk(cuda, [5 * T + 7, 700, 33, 0, 16 * T], [40, 130, 33, 0, 1], 2, T, D, 4, window=window, sinks=sinks, seed=T + D)
        encode(c, kv, amax, PATTERNS[pattern])
        check(c, c.run(kv), lambda b, n: (c.starts[b] + np.arange(c.new[b]), n - c.new[b] + np.arange(c.new[b])))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_and_joined(kv, cuda, D):
    """Over all SMs: parts that lie in pages without a value beside parts that do not; all pages empty; all scales 1."""
    for lens, zero in (([9000], lambda b, j: j < 40), ([9000], lambda b, j: 30 < j), ([5000, 700], lambda b, j: True), ([9000], lambda b, j: False)):
        c = Cache(cuda, "fp8", lens, 1, 64, D, 4, seed=1)
        encode(c, kv, 1e-5, zero)
        check(c, c.run(kv), lambda b, n: ([b], [n - 1]))
        e = Chunk(cuda, lens, [40] * len(lens), 1, 64, D, 4, seed=1)
        encode(e, kv, 1e-5, zero)
        rows = lambda b, n: (40 * b + np.arange(40), n - 40 + np.arange(40))  # noqa: E731
        check(e, e.run(kv), rows)
        for x in (c, e):   # the same codes with scales of 1: some tiles of zeros, most not
            x.kb, x.vb = torch.full_like(x.kb, 0.01), torch.ones_like(x.vb)
        check(c, c.run(kv), lambda b, n: ([b], [n - 1]))
        check(e, e.run(kv), rows)


def test_hidden_tokens_do_not_count_as_values(kv, cuda):
    """A page whose visible tokens are all 0 and whose hidden ones are not (the last, and one at a window's begin)."""
    for make, rows in ((lambda: Cache(cuda, "fp8", [330], 1, 64, 128, 4, 100, 0, seed=2), lambda b, n: ([0], [n - 1])),
                       (lambda: Chunk(cuda, [330], [1], 1, 64, 128, 4, window=100, sinks=0, seed=2), lambda b, n: ([0], [n - 1]))):
        c = make()
        encode(c, kv, 1e-5, lambda b, j: j in (3, 5))
        # window: tokens 230 .. 329; pages 3 (192 .. 255) and 5 (320 .. 383)
        c.v[c.table[0, 3], :, :32] = 0x70
        c.v[c.table[0, 5], :, 10:] = 0x70
        check(c, c.run(kv), rows)
