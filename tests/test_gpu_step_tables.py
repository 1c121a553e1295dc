"""Page tables and slots of a step against plain loops over Python integers: every output equal."""
import random

import pytest
import torch

import plain_windows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


class Step:
    """A step's arrays on the host: requests with tables out of one pool, and a stack of the pages that are free."""

    def __init__(self, seed, B, T, maxp, free, past=None, new=None, rows=None, spare=0, slack=3):
        r = random.Random(seed)
        self.T, self.maxp = T, maxp
        self.past = [r.randint(0, maxp * T) if r.random() < 0.9 else 0 for _ in range(B)] if past is None else list(past)
        room = [maxp * T - p for p in self.past]
        self.new = [min(room[b], r.choice((-1, 0, 1, 1, r.randint(0, 3 * T)))) for b in range(B)] if new is None else list(new)
        have = [max(0, -(-p // T)) for p in self.past]
        ids = list(range(sum(have) + free))
        r.shuffle(ids)
        self.table = [[-7] * maxp for _ in range(B)]
        for b, n in enumerate(have):
            for j in range(min(n, maxp)):
                self.table[b][j] = ids.pop()
        self.stack, self.count = ids + [-9] * (sum(have) + spare), len(ids)
        self.rows = sum(max(a, 0) for a in self.new) + slack if rows is None else rows
        self.full_cap = B + self.rows // T + 2

    def want(self):
        return plain_windows.step_tables(self.past, self.new, self.stack, self.count, self.table, self.T, self.rows, self.full_cap)

    def to(self, dev):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        B = len(self.past)
        z = lambda n, t=torch.int32: torch.full((n,), 99, dtype=t, device=dev)  # noqa: E731
        self.t = {"past": i(self.past), "new": i(self.new), "stack": i(self.stack), "count": i([self.count]), "table": i(self.table),
                  "lens": z(B), "starts": z(B + 1), "slots": z(self.rows, torch.int64), "positions": z(self.rows),
                  "full": z(self.full_cap), "left": z(1), "status": torch.zeros(1, dtype=torch.int32, device=dev)}
        return self

    def run(self, kv, inplace=False, **kw):
        t = self.t
        if inplace:
            t["lens"], t["left"] = t["past"], t["count"]
        kv.nvfp4_kv_step_tables(kv.Layout(1, 64, self.T), t["past"], t["new"], t["stack"], t["count"], t["table"], t["lens"],
                                t["starts"], t["slots"], t["positions"], free_left=None if inplace else t["left"],
                                full_pages=t["full"], status=t["status"], **kw)

    def check(self):
        want = self.want()
        for name, x in want.items():
            got = self.t[name].cpu().tolist()
            assert (got if isinstance(x, list) else got[0]) == x, (name, got if len(str(got)) < 400 else "", x if len(str(x)) < 400 else "")
        return want


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,T,maxp,free", [(1, 16, 1, 3), (3, 64, 7, 40), (40, 16, 9, 300), (1025, 48, 5, 3000), (3000, 1, 6, 9000),
                                           (8192, 16, 2, 9000)])
def test_steps(kv, cuda, B, T, maxp, free, inplace):
    s = Step(B + T, B, T, maxp, free).to(cuda)
    s.run(kv, inplace)
    assert s.check()["status"] == 0


@pytest.mark.parametrize("seed", range(6))
def test_few_pages_beside_those_given_back(kv, cuda, seed):
    s = Step(seed, 300, 16, 12, 15 * seed, spare=5).to(cuda)
    s.run(kv)
    s.check()


@pytest.mark.parametrize("seed", range(6))
def test_too_few_pages(kv, cuda, seed):
    """Some are served, some not; those that need no page are."""
    s = Step(seed, 300, 16, 12, 15 * seed, spare=5)
    s = Step(seed, 300, 16, 12, 15 * seed, spare=5, past=s.past, new=[max(a, 0) for a in s.new]).to(cuda)
    s.run(kv)
    assert s.check()["status"] == plain_windows.NO_PAGES


def test_more_pages_given_back_than_the_stack_holds(kv, cuda):
    s = Step(1, 50, 16, 8, 4)
    s.stack = s.stack[:s.count + 20]
    s.to(cuda).run(kv)
    assert s.check()["status"] & plain_windows.PAGE_OOB


@pytest.mark.parametrize("count", [-5, 1000])
def test_a_count_outside_the_stack(kv, cuda, count):
    s = Step(2, 20, 16, 8, 400)
    s.stack, s.count = s.stack[:420] if count < 0 else [i % 300 for i in range(420)], count
    s.to(cuda).run(kv)
    assert s.check()["status"] & plain_windows.PAGE_OOB


def test_bad_lengths_and_rows_that_do_not_fit(kv, cuda):
    big = 2 ** 31 - 1
    s = Step(3, 0, 16, 4, 60, past=[], new=[])
    past, new = [5, -1, 64, 65, 10, big, 3, -big, 0, 7, 9], [3, 4, 1, 0, big, 2, -2, -1, 20, 4, 30]
    s = Step(3, 11, 16, 4, 60, past=[max(0, min(p, 64)) for p in past], new=new, rows=40)
    s.past = past
    s.to(cuda).run(kv)
    want = s.check()
    assert want["status"] == plain_windows.BAD_SEQ_LEN and want["lens"] == [8, 0, 64, 0, 10, 0, 3, 0, 0, 7, 9]
    # and with rows enough for all but the one that adds 2^31 - 1 tokens
    s = Step(3, 3, 16, 4, 60, past=[5, 0, 7], new=[3, big, 4], rows=100).to(cuda)
    s.run(kv)
    assert s.check()["starts"] == [0, 3, 100, 100]


@pytest.mark.parametrize("rows", [0, 1, 5])
def test_few_rows_and_nothing_to_do(kv, cuda, rows):
    s = Step(4, 7, 16, 4, 9, new=[0] * 7, rows=rows).to(cuda)
    if rows == 0:   # an empty tensor has no address: the C call takes it as left out
        s.full_cap = 9
    s.run(kv)
    s.check()


def test_all_requests_end_and_others_take_their_pages(kv, cuda):
    past = [40, 33, 16, 0, 1, 64]
    s = Step(5, 6, 16, 5, 0, past=past, new=[-1, 20, -1, 30, -1, -1]).to(cuda)
    s.run(kv)
    want = s.check()
    assert want["status"] == 0 and set(want["table"][3][:2]) <= set(sum(s.table, []))


def test_many_steps_in_place_and_as_a_graph(kv, cuda):
    """A decode loop of 40 steps as replays of one graph over lengths, stack and tables that stay in place: tables hold
    each page once, and every token has the slot that its table says."""
    B, T, maxp = 9, 16, 8
    s = Step(6, B, T, maxp, B * maxp, past=[0] * B, new=[3, 1, 1, 1, 1, 0, 2, 1, 1]).to(cuda)
    s.run(kv, inplace=True)   # (the first call sets the attribute of the kernel)
    past, stack, count, table = s.want()["lens"], s.want()["stack"], s.want()["left"], s.want()["table"]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        s.run(kv, inplace=True)
    for _ in range(40):
        graph.replay()
        s.past, s.stack, s.count, s.table = past, stack, count, table
        want = s.want()
        s.t["status"].zero_()
        for name in ("lens", "starts", "slots", "positions", "full", "table", "stack"):
            assert s.t[name].cpu().tolist() == want[name], name
        past, stack, count, table = want["lens"], want["stack"], want["left"], want["table"]
    live = [p for b in range(B) for p in table[b][:-(-past[b] // T)]]
    assert len(live) == len(set(live)) and set(live).isdisjoint(stack[:count])
