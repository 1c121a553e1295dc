"""The ring of places through which the extend attention's scout tells the other warps of a block where their KV tiles lie, as a
model: warps step in any order, and at some moment a wait gives up, after which none waits. Whatever is read must then still be
in bounds, and every warp must come to an end. (csrc/extend_attention.cu: warp_wait, scout_tiles, load_tiles, softmax_rows.)"""
import random

import pytest

RING, GROUPS, ROWS, NO_ROW = 8, 3, 100, 2 ** 32 - 1
FULL, LAST, END, OVER = 1, 2, 4, 8
GARBAGE = 2 ** 31


class Block:
    """`mended` False: as before places were initialised, groups without a page marked in the flags, and the scout stopped."""

    def __init__(self, seed, tiles, mended=True):
        r = self.r = random.Random(seed)
        self.mended, self.tiles = mended, tiles
        first = dict(flags=OVER | LAST | END, rows=[0] * GROUPS, y=0, z=0) if mended else dict(flags=0, rows=[GARBAGE] * GROUPS, y=GARBAGE, z=GARBAGE)
        self.ring = [dict(first, rows=list(first["rows"])) for _ in range(RING)]
        # (a piece is a run of tiles of one unit, whose rows are z .. z + y)
        self.places, left = [], 0
        for n in range(tiles):
            if left == 0:
                left, z = r.randint(1, 9), r.randint(0, ROWS - 1)
                y = r.randint(1, ROWS - z)
            left -= 1
            rows = [r.randint(0, 999) if r.random() < 0.7 else None for _ in range(GROUPS)]
            last = left == 0 or n + 1 == tiles
            flags = (FULL if None not in rows else 0) | (LAST if last else 0) | (END if n + 1 == tiles else 0)
            self.places.append((flags | sum(16 << g for g in range(GROUPS) if rows[g] is None), rows, y, z))
        self.placed = self.loaded = 0
        self.done = {}
        self.dead = False
        self.faults = []

    def wait(self, ready):
        while not (self.dead or ready()):
            yield

    def scout(self):
        for n, (flags, rows, y, z) in enumerate(self.places):
            if n >= RING:
                yield from self.wait(lambda: self.loaded >= n - (RING - 3))
                if self.mended and self.dead:
                    for d in self.ring:
                        d["flags"] = OVER | LAST | END
                        yield
                    return
            d = self.ring[n % RING]
            words = [("rows", g) for g in range(GROUPS)] + ["flags", "y", "z"]
            self.r.shuffle(words)
            for w in words:  # (the order that the memory sees them in: any)
                if w == "flags":
                    d["flags"] = flags
                elif isinstance(w, tuple):
                    d["rows"][w[1]] = rows[w[1]] if rows[w[1]] is not None else 0 if self.mended else NO_ROW
                else:
                    d[w] = y if w == "y" else z
                yield
            self.placed = n + 1

    def loader(self, name, first):
        n = 0
        while True:
            yield from self.wait(lambda: self.placed > n)
            d = self.ring[n % RING]
            flags = d["flags"]
            if flags & OVER:
                return
            for g in range(GROUPS):
                yield
                row = d["rows"][g]
                if not flags & FULL and (flags >> (4 + g) & 1 if self.mended else row == NO_ROW):
                    continue
                if row >= 1000:
                    self.faults.append((name, n, row))
            yield from self.wait(lambda: self.done["softmax"] >= n - 1)
            self.done[name] = n + 1
            if first:
                self.loaded = n + 1
            yield
            if flags & END:
                return
            n += 1

    def softmax(self):
        n, begins = 0, True
        while True:
            yield from self.wait(lambda: self.placed > n)
            d = self.ring[n % RING]
            if begins:
                flags = d["flags"]
                if flags & OVER and n == 0:
                    return
                if not flags & OVER:
                    yield
                    y = d["y"]
                    yield
                    z = d["z"]
                    for t in (0, y - 1):
                        if 0 <= t < y and (z + t < ROWS or not self.mended) and not 0 <= z + t < ROWS:
                            self.faults.append(("softmax", n, z + t))
            yield from self.wait(lambda: all(v > n for k, v in self.done.items() if k != "softmax"))
            flags = d["flags"]
            yield
            n += 1
            self.done["softmax"] = n
            begins = bool(flags & LAST)
            if begins and flags & END:
                return

    def run(self, gives_up):
        """-> the faults, or None where a warp does not end."""
        roles = {"scout": self.scout(), "softmax": self.softmax()}
        for i in range(3):
            roles[f"load{i}"] = self.loader(f"load{i}", i == 0)
        self.done = {k: 0 for k in roles if k != "scout"}
        speed = {k: self.r.random() ** 2 + 0.02 for k in roles}
        for step in range(60000):
            if not roles:
                return self.faults
            if step == gives_up:
                self.dead = True
            k = self.r.choices(list(roles), [speed[k] for k in roles])[0]
            if next(roles[k], "end") == "end":
                del roles[k]
        return None


@pytest.mark.parametrize("seed", range(300))
def test_after_a_wait_gave_up(seed):
    tiles = random.Random(seed).choice((1, 3, 9, 40))
    assert Block(seed, tiles).run(gives_up=random.Random(-seed).randint(0, 40 * tiles)) == []


@pytest.mark.parametrize("seed", range(30))
def test_without_one(seed):
    for mended in (True, False):
        assert Block(seed, 40, mended).run(gives_up=None) == []


def test_the_model_finds_what_it_is_for():
    """Without initialised places, marked groups and a scout that stops, something is read out of bounds or goes on for ever."""
    bad = [Block(seed, 9, mended=False).run(gives_up=random.Random(-seed).randint(0, 360)) for seed in range(100)]
    assert sum(b is None or b != [] for b in bad) > 20
