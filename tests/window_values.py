"""The decode caches of test_gpu_window_decode with values whose averages stay large over many tokens, held to bounds with the
largest |v| that a sequence's tokens have."""
import numpy as np
import torch

import plain_windows
from test_gpu_window_decode import Cache


class Leaning(Cache):
    """V above 0 in the even dims and below in the odd ones, scores 1.6 times as far apart: the outputs are a fifth of the largest
    |v| and more, and the heads differ."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        odd = torch.arange(self.D) % 2 == 1
        if self.fmt == "fp8":
            self.v = (self.v & 0x7F) | torch.where(odd, 0x80, 0).to(torch.uint8)
        else:
            self.vd = (self.vd & 0x77) | torch.where(odd, 0x88, 0).to(torch.uint8)
        self.sm = float(np.float32(1.6 * self.sm))
        self.parts = list(parts(self))


def parts(c):
    """(sequence, KV head, its q rows, k, v, visible) of every pair that sees a token."""
    for b, n in enumerate(c.lens):
        for h in range(c.H):
            k, v, ok = c.tokens(b, h)
            here = np.repeat(plain_windows.visible([n - 1], n, c.window, c.sinks) & ok, c.G, 0) if n else np.zeros((c.G, 0), bool)
            if here.any():
                yield b, slice(h * c.G, (h + 1) * c.G), c.q[b, h * c.G:(h + 1) * c.G].double().numpy(), k, v, here


def check(c, got):
    out, lse = got
    for b, heads, q, k, v, here in c.parts:
        plain_windows.check((out[b, heads], lse[b, heads]), q, k, v, here, c.sm, np.abs(v[here.any(0)]).max(), blocks=c.fmt == "fp8")


def exact(c, drop=None):
    """out, lse of every pair in 64 bits; with `drop` = n the heaviest of n parts of the visible tokens is left out of out."""
    out, lse = np.zeros(c.q.shape), np.full(tuple(c.q.shape[:2]), -np.inf)
    for b, heads, q, k, v, here in c.parts:
        out[b, heads], lse[b, heads] = plain_windows.attention(q, k, v, here, c.sm)
        if drop:
            at = np.array_split(np.flatnonzero(here.any(0)), drop)
            w = [np.exp(q @ k[a].T * c.sm - lse[b, heads, None]) for a in at]
            i = int(np.argmax([x.sum() for x in w]))
            out[b, heads] -= w[i] @ v[at[i]]
    return out, lse


LONG = [([40000], 39000, 0), ([9000, 30011], 20000, 300), ([70001], 6000, 40)]
