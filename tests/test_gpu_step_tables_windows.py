"""Step tables of sequences that gave pages back before they ended (a sliding window): entries below 0 are not pages."""
import random

import pytest
import torch

import plain_windows
from test_gpu_step_tables import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


class Holes(Step):
    """What is wanted is the plain form's result for ended sequences that never had the missing pages. A row whose page is
    not one has no slot."""

    def want(self):
        past, table = list(self.past), [list(r) for r in self.table]
        for b, (n, a) in enumerate(zip(self.past, self.new)):
            if a == -1 and 0 <= n <= self.maxp * self.T:
                kept = [e for e in self.table[b][:-(-n // self.T)] if e >= 0]
                past[b], table[b] = len(kept) * self.T, (kept + [-1] * self.maxp)[:self.maxp]
        w = plain_windows.step_tables(past, self.new, self.stack, self.count, table, self.T, self.rows, self.full_cap)
        for b, a in enumerate(self.new):
            if a == -1:
                w["table"][b] = list(self.table[b])
        at = 0
        for b, a in enumerate(self.new):
            for r in range(at, min(at + max(a, 0), self.rows)):
                served = w["lens"][b] == self.past[b] + a
                if served and w["table"][b][(self.past[b] + r - at) // self.T] < 0:
                    w["slots"][r], w["positions"][r] = -1, 0
                    w["status"] |= plain_windows.PAGE_OOB
            at += max(a, 0)
        return w

    def drop(self, gone):
        """Entries j of sequence b with gone(b, j, pages) become ids that are no page."""
        for b, n in enumerate(self.past):
            have = -(-n // self.T)
            for j in range(have):
                if gone(b, j, have):
                    self.table[b][j] = -1 - 1000 * (j % 3)
        return self


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,T,maxp,free", [(5, 16, 60, 40), (40, 16, 200, 9), (1025, 48, 9, 0), (3000, 1, 6, 100), (8192, 16, 3, 9000)])
def test_windows_that_ended(kv, cuda, B, T, maxp, free, inplace):
    """The first page and the last two are left: their pages go on the stack and to the others, the missing ones to nobody."""
    s = Holes(B, B, T, maxp, free, spare=3).drop(lambda b, j, n: 1 <= j < n - 2)
    s.to(cuda).run(kv, inplace)
    want = s.check()
    assert min(want["stack"][:want["left"]], default=0) >= 0 and want["status"] & plain_windows.PAGE_OOB == 0


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("seed", range(8))
def test_any_entries_missing(kv, cuda, seed, inplace):
    """Missing at random: a few, half, nearly all, all; also of sequences that go on, whose last pages are there."""
    r = random.Random(seed)
    share = (0.02, 0.5, 0.95, 1.0)[seed % 4]
    s = Holes(seed, 300, 16, 40, 200 if seed < 4 else 0, spare=2)
    s.drop(lambda b, j, n: r.random() < share and (s.new[b] == -1 or j < n - 1))
    s.to(cuda).run(kv, inplace)
    s.check()


def test_a_sequence_that_ended_beside_one_that_grows(kv, cuda):
    """Table [3, -1, -1, -1, 7] ends: pages 3 and 7 are free, and the other sequence, which needs three, is not served with
    two; with one more on the stack it is, and no page is dealt twice."""
    for extra in (0, 1):
        s = Holes(0, 2, 16, 5, 0, past=[70, 0], new=[-1, 40])
        s.table = [[3, -1, -1, -1, 7], [-7] * 5]
        s.stack, s.count = [9] * extra + [-9] * 6, extra
        s.to(cuda).run(kv)
        want = s.check()
        if extra:
            assert want["status"] == 0 and want["table"][1][:3] == [7, 3, 9] and min(want["slots"][:40]) >= 0 and want["left"] == 0
        else:
            assert want["status"] == plain_windows.NO_PAGES and want["left"] == 2 and want["stack"][:2] == [3, 7]


def test_long_rows_with_few_pages(kv, cuda):
    """131072 tokens of which a window left 5 and 65 pages, several of them, with room for all that comes back."""
    s = Holes(1, 12, 64, 2050, 100, past=[131072 - 17 * b for b in range(12)], new=[-1, 3, -1, -1, 1, -1, 64, -1, 1, -1, -1, 200])
    s.drop(lambda b, j, n: 5 <= j < n - 65).to(cuda).run(kv)
    assert s.check()["status"] == 0


def test_ids_that_are_no_page_give_no_slot(kv, cuda):
    """Ids below 0 on the stack, and a cached page that is partly filled and was given back: slot -1, PAGE_OOB."""
    s = Holes(2, 3, 16, 4, 0, past=[5, 16, 30], new=[3, 20, 1])
    s.table = [[-1, -7, -7, -7], [4, -7, -7, -7], [1, 2, -7, -7]]
    s.stack, s.count = [6, -1, -5, 8], 4
    s.to(cuda).run(kv)
    want = s.check()
    assert want["status"] == plain_windows.PAGE_OOB and want["slots"][:3] == [-1] * 3 and want["table"][1][1:3] == [8, -5]
    assert want["slots"][3:19] == list(range(128, 144)) and want["slots"][19:23] == [-1] * 4 and want["slots"][23] == 46


def test_captured(kv, cuda):
    """A graph replayed as windows move on: sequences end with holes in place, others take their pages."""
    B, T, maxp = 6, 16, 40
    s = Holes(3, B, T, maxp, 90, past=[600, 300, 0, 17, 400, 64], new=[-1, 20, 33, -1, 1, 1]).drop(lambda b, j, n: 1 <= j < n - 2)
    s.to(cuda).run(kv, inplace=True)
    s.check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        s.run(kv, inplace=True)
    for new in ([5, -1, 1, 40, -1, 1], [1, 7, -1, 1, 2, -1]):
        now = s.want()
        s.past, s.stack, s.count, s.table, s.new = now["lens"], now["stack"], now["left"], now["table"], list(new)
        s.rows = s.t["slots"].shape[0]
        s.drop(lambda b, j, n: 2 <= j < n - 3)
        for name, x in (("table", s.table), ("new", s.new)):
            s.t[name].copy_(torch.tensor(x, dtype=torch.int32))
        s.t["status"].zero_()
        graph.replay()
        s.check()
