"""NaN in keys, values and page scales of the extend attention: it reaches the rows that see it, in the dims that it has, and no
others, whatever tile and unit they share."""
import numpy as np
import pytest
import torch

import plain_windows
from test_gpu_extend_attention import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


CASES = [([5], [5], 16, 0, 0), ([170, 300, 37], [20, 7, 37], 32, 0, 0), ([170, 300, 37], [90, 130, 37], 16, 40, 3), ([700], [400], 64, 0, 0),
         ([700, 333], [300, 333], 48, 129, 70), ([4000, 64], [150, 1], 64, 0, 0), ([4000], [150], 64, 1000, 200)]


def seen(c, b):
    """[rows, tokens] of sequence b: which tokens its rows see."""
    n, m = c.lens[b], c.new[b]
    return plain_windows.visible(n - m + np.arange(m), n, c.window, c.sinks)


def places(c, seed, per=7):
    """Tokens of each sequence: the chunk's last and first, its borders, the window's begin, and any."""
    r = np.random.default_rng(seed)
    for b, (n, m) in enumerate(zip(c.lens, c.new)):
        at = {n - 1, n - m, n - m // 2 - 1, max(0, n - m - 1), max(0, n - (c.window or n) - 1)} | set(r.integers(0, n, per).tolist())
        for t in sorted(at):
            page = int(c.table[b, t // c.T])
            if 0 <= page < c.P:
                yield b, t, page


def same(a, b):
    return np.array_equal(a[~np.isnan(b)], b[~np.isnan(b)]) and np.isnan(a[np.isnan(b)]).all()


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (256, 3), (128, 7)])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("blocks", [True, False])
def test_values(kv, cuda, D, G, case, blocks):
    lens, new, T, window, sinks = CASES[case]
    c = Chunk(cuda, lens, new, 2, T, D, G, window=window, sinks=sinks, seed=case, blocks=blocks, padding=3)
    r = np.random.default_rng(case)
    marks = [(b, t, page, int(r.integers(2)), int(r.integers(D)), int(r.choice((0x7F, 0xFF)))) for b, t, page in places(c, case)]
    for b, t, page, h, d, _ in marks:
        c.v[page, h, t % T, d] = 0
    want = c.run(kv)
    out = want[0].copy()
    for b, t, page, h, d, _ in marks:
        rows = c.starts[b] + np.flatnonzero(seen(c, b)[:, t])
        out[rows, h * G:(h + 1) * G, d] = np.nan
    for b, t, page, h, d, code in marks:
        c.v[page, h, t % T, d] = code
    got = c.run(kv)
    assert np.isfinite(out[:c.starts[-1]]).sum() and np.isnan(out[:c.starts[-1]]).any()
    assert same(got[0], out) and same(got[1], want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["keys", "k scale", "v scale", "infinite scale"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_keys_and_scales(kv, cuda, D, what, case):
    """One key, or one page's scale, of a head: the rows that see the token, or a token of the page, are NaN in all dims."""
    lens, new, T, window, sinks = CASES[case]
    G = 4
    c = Chunk(cuda, lens, new, 2, T, D, G, window=window, sinks=sinks, seed=case, padding=2)
    want = c.run(kv)
    for b, t, page in list(places(c, case, per=1)):
        h = t % 2
        keep = c.k.clone(), c.kb.clone(), c.vb.clone()
        if what == "keys":
            c.k[page, h, t % T, 3 * t % D] = 0xFF
            hit = seen(c, b)[:, t]
        else:
            (c.kb if what == "k scale" else c.vb)[page, h] = float("inf" if what == "infinite scale" else "nan")
            j = t // T
            hit = seen(c, b)[:, j * T:(j + 1) * T].any(1)
        got = c.run(kv)
        rows = c.starts[b] + np.flatnonzero(hit)
        heads = slice(h * G, (h + 1) * G)
        assert np.isnan(got[0][rows, heads]).all()
        for x, y in zip(got, want):
            x[rows, heads] = y[rows, heads]
            assert np.array_equal(x, y, equal_nan=True)
        c.k, c.kb, c.vb = keep
