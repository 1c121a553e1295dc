"""Plain 64-bit forms of the step tables, the FP8 pages and the attentions over FP8 pages and with a sliding window,
written from their definitions with numpy and loops, and the bound that the attentions' outputs are held to."""
import numpy as np

import plain_steps

LOG2E = 1.4426950408889634
# E4M3 byte -> value (the two NaN bytes as NaN)
FP8 = np.array([s * (m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) if (e, m) != (15, 7) else np.nan
                for s in (1, -1) for e in range(16) for m in range(8)])
BAD_SEQ_LEN, PAGE_OOB, NO_PAGES = 0x2, 0x1, 0x10


def step_tables(past, new, stack, count, table, T, rows, full_cap):
    """Everything as lists of Python integers; returns a dict of what the call writes, with its status bits."""
    B, maxp, cap = len(past), len(table[0]), len(stack)
    table, stack, status = [list(r) for r in table], list(stack), 0
    pages = lambda n: -(-n // T)  # noqa: E731
    if not 0 <= count <= cap:
        status |= PAGE_OOB
        count = max(0, min(count, cap))
    good = [0 <= p <= maxp * T and a >= -1 and p + max(a, 0) <= maxp * T for p, a in zip(past, new)]
    top = count
    for b in range(B):
        if good[b] and new[b] == -1:
            for j in range(pages(past[b])):
                if top < cap:
                    stack[top] = table[b][j]
                    top += 1
                else:
                    status |= PAGE_OOB
    asked = taken = row = 0
    lens, starts, slots, positions, full = [], [], [-1] * rows, [0] * rows, []
    for b in range(B):
        p, a = past[b] if 0 <= past[b] <= maxp * T else 0, new[b]
        n = max(a, 0)
        starts.append(min(row, rows))
        need = pages(p + n) - pages(p) if good[b] else 0
        asked += need
        ok = good[b]
        if not ok or (n > 0 and row + n > rows):
            status |= BAD_SEQ_LEN
            ok = False
        elif need and asked > top:
            status |= NO_PAGES
            ok = False
        if not ok:
            lens.append(p)
        elif a == -1:
            lens.append(0)
        else:
            for j in range(need):
                table[b][pages(p) + j] = stack[top - 1 - taken]
                taken += 1
            for i in range(n):
                slots[row + i] = table[b][(p + i) // T] * T + (p + i) % T
                positions[row + i] = p + i
            full += [table[b][j] for j in range(p // T, (p + n) // T)]
            lens.append(p + n)
        row += n
    starts.append(min(row, rows))
    return {"lens": lens, "starts": starts, "slots": slots, "positions": positions, "full": (full + [-1] * full_cap)[:full_cap],
            "left": top - taken, "table": table, "stack": stack, "status": status}


def fp8_encode(x):
    """Bytes of E4M3_rne_satfinite of x (in FP32)."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    return (plain_steps.nearest(a, plain_steps.E4M3) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def fp8_page(x, tokens):
    """x [H, T, D]: bytes and scales [H]."""
    x = np.array(x, dtype=np.float64)
    x[:, tokens:] = 0
    f32 = plain_steps.f32
    s = f32(np.abs(x).max((1, 2)) / 448)
    s = np.where(s < 2.0 ** -100, 1.0, s)
    code = fp8_encode(f32(x * f32(1 / s)[:, None, None]))
    code[:, tokens:] = 0
    return code, s


def visible(pos, n, window, sinks):
    """[rows, n]: which of n tokens the rows at these positions see."""
    t, p = np.arange(n)[None], np.asarray(pos)[:, None]
    return (t <= p) & ((t > p - window) | (t < sinks)) if window else t <= p


def attention(q, k, v, here, scale):
    """q [rows, D] over k, v [n, D], of which the row sees here [rows, n]: out, lse."""
    x = np.where(here, q @ k.T * scale, -np.inf)
    top = x.max(-1, keepdims=True, initial=-np.inf)
    some = top > -np.inf
    p = np.where(here, np.exp(x - np.where(some, top, 0)), 0.0)
    total = p.sum(-1, keepdims=True)
    out = p @ np.where(here.any(0)[:, None], v, 0.0) / np.where(some, total, 1)
    return out, np.where(some, top + np.log(np.where(some, total, 1)), -np.inf)[:, 0]


def check(got, q, k, v, here, scale, vmax, blocks=False, logs=20):
    """Rows of out [rows, D] and lse [rows] against 64 bits. With x a token's score in log2 units the kernels round

      x     a sum of D exact products in FP32 (2^-23 of sum |products| for each of the D additions), its product with
            the scale (2^-24 |x|), and the scale itself (3 2^-24 |x|, alike for all tokens of a head). With scales of
            pages: the page's scale (2^-24 |x|), and log2 of V's, which is added (2^-22 of its approximation, at most 2^-22
            of its size, and 2^-24 of the sum) and whose inverse counts in the sum of weights (2^-22)
      p     2^-22 (the approximate 2^y), then, before P V, to FP16: 2^-11, and 2^-25 where p is subnormal (against a
            largest p of at least 2^-1)
      sums  FP32: 2^-23 of sum |terms| for each of n additions, 2^-21 for a join
      out   to BF16: half a step

    so |out - exact| <= half a step + A (2^-11 + 2 (2^-22 + dx + 2^-23 n) + 2^-21) + 2^-24 n vmax, A = sum of weight |v|,
    dx what two scores may move apart (|log2 s| <= logs) and vmax the largest E4M3 (or E2M1 E4M3) value times the largest scale."""
    out, lse = got
    want, want_lse = attention(q, k, v, here, scale)
    assert np.isfinite(out).all()
    none = ~here.any(-1)
    assert (out[none] == 0).all() and (lse[none] == -np.inf).all()
    some = ~none
    if not some.any():
        return
    out, lse, want, want_lse, here, q = out[some], lse[some], want[some], want_lse[some], here[some], q[some]
    k, v = np.where(here.any(0)[:, None], k, 0.0), np.where(here.any(0)[:, None], v, 0.0)
    x = q @ k.T * scale
    w = np.where(here, np.exp(np.where(here, x - want_lse[:, None], -np.inf)), 0.0)
    A = w @ np.abs(v)
    D = q.shape[1]
    S = np.where(here, np.abs(q) @ np.abs(k).T, 0.0).max(-1) * abs(scale) * LOG2E
    big = np.where(here, np.abs(x), 0.0).max(-1) * LOG2E
    dist = (np.where(here, x, -np.inf).max(-1) - np.where(here, x, np.inf).min(-1)) * LOG2E
    dx = 2.0 ** -24 * (2 * big + 3 * dist) + 2 * 2.0 ** -23 * D * S
    if blocks:
        dx = dx + 2 * (2.0 ** -24 * 2 * (big + logs) + 2 * 2.0 ** -22 * logs + 2.0 ** -22)
    dx = (np.log(2) * dx)[:, None]
    n = here.sum(-1)[:, None]
    rel = 2.0 ** -11 + 2 * (2.0 ** -22 + dx + 2.0 ** -23 * n) + 2.0 ** -21
    tol = A * rel + 2.0 ** -24 * n * vmax
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want) + tol, 2.0 ** -126))) - 8)
    err = np.abs(out - want)
    assert (err <= tol + half).all(), (float((err - tol - half).max()), float(err.max()), np.argwhere(err > tol + half)[:5])
    ltol = 2.0 ** -24 * 7 * np.maximum(big, np.abs(want_lse) * LOG2E) + dx[:, 0] + 2.0 ** -22 * n[:, 0] + 2.0 ** -20
    assert (np.abs(lse - want_lse) <= ltol).all(), (np.abs(lse - want_lse).max(), ltol.min())
