"""Plain 64-bit forms of the decode-step operators (append with rotation, page bounds, page selection,
attention over selected pages), written from their definitions with numpy and loops; every FP32
rounding of a definition is an FP64 operation rounded to FP32 (exact: 53 >= 2 * 24 + 2)."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)][:127])


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def nearest(y, grid):
    """Index of the grid value nearest to y >= 0 (ties to the even index, saturating at the top)."""
    y = np.minimum(np.asarray(y, dtype=np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, y), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - y, y - grid[lo]
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def rotate(x, row, style, first, dims):
    """x [heads, D] rotated by the table row (cosines, then sines)."""
    x = np.array(x, dtype=np.float64)
    half = dims // 2
    i = np.arange(half)
    one, two = (first + i, first + half + i) if style == "halves" else (first + 2 * i, first + 2 * i + 1)
    c, s = np.asarray(row[:half], dtype=np.float64), np.asarray(row[half:], dtype=np.float64)
    a, b = x[:, one].copy(), x[:, two].copy()
    x[:, one] = f32(f32(a * c) - f32(b * s))
    x[:, two] = f32(f32(b * c) + f32(a * s))
    return x


def encode(x, g):
    """Codes [.., D] (0..15) and scale bytes [.., D/16] of x [.., D]."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 16)
    g = float(g)
    sb = nearest(f32(np.abs(b).max(-1) / f32(6 * g)), E4M3)
    sg = f32(E4M3[sb] * g)
    r = np.where(sg > 0, f32(1 / np.where(sg > 0, sg, 1)), 0.0)[..., None]
    y = f32(b * r)
    code = nearest(np.abs(y), E2M1) | np.where(np.signbit(y), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def decode(code, sb, g):
    """fp32(e2m1 * e4m3 * g) of codes [.., D] and scale bytes [.., D/16]."""
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = v.reshape(*code.shape[:-1], -1, 16) * E4M3[sb][..., None]
    return f32(v * float(g)).reshape(code.shape)


def append(pool, k, v, slots, T, g_k, g_v, rot=None, positions=None, q=None):
    """Append rows to the numpy pools {kd, ks, vd, vs} in place; rows with a bad slot or position are
    skipped. Returns the rotated q, and k and v as stored, as lists of [heads, D] or None per row.
    rot = (style, first, dims, table)."""
    P = pool["kd"].shape[0]
    qs, ks, vs = [], [], []
    for n, s in enumerate(np.asarray(slots)):
        ok = 0 <= s < P * T
        if ok and rot is not None:
            ok = 0 <= positions[n] < rot[3].shape[0]
        if not ok:
            qs.append(None), ks.append(None), vs.append(None)
            continue
        page, t = int(s) // T, int(s) % T
        turn = (lambda x: rotate(x, rot[3][positions[n]], *rot[:3])) if rot is not None else \
            (lambda x: np.array(x, dtype=np.float64))
        qs.append(None if q is None else turn(q[n]))
        code, sb = encode(turn(k[n]), g_k)
        pool["kd"][page, :, t] = code[:, 0::2] | (code[:, 1::2] << 4)
        pool["ks"][page, :, t] = sb
        ks.append(decode(code, sb, g_k))
        code, sb = encode(np.array(v[n], dtype=np.float64), g_v)
        old = pool["vd"][page, :, t // 2]
        pool["vd"][page, :, t // 2] = (old & 0xF0) | code if t % 2 == 0 else (old & 0x0F) | (code << 4)
        pool["vs"][page, :, t // 2, :, t % 2] = sb
        vs.append(decode(code, sb, g_v))
    return qs, ks, vs


def keys(kd, ks):
    """K values without g: codes [.., T, D/2] and scale bytes [.., T, D/16] to [.., T, D]."""
    code = np.stack([kd & 15, kd >> 4], -1).reshape(*kd.shape[:-1], -1)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    # a NaN scale byte (0x7F) gets 0: only tokens that must not count may hold one
    sc = np.append(E4M3, 0.0)[ks & 127] * np.where(ks & 128, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, 16) * sc[..., None]).reshape(v.shape)


def page_bounds(kd, ks, tokens):
    """hi, lo [H, D] and scale [H] of one page (kd [H, T, D/2])."""
    H, D = kd.shape[0], kd.shape[2] * 2
    if tokens == 0:
        return np.zeros((H, D), np.int8), np.zeros((H, D), np.int8), np.zeros(H, np.float32)
    v = keys(kd, ks)[:, :tokens]
    top, low = v.max(1), v.min(1)
    s = f32(np.maximum(np.abs(top), np.abs(low)).max(-1) / 127)
    d = np.where(s > 0, s, 1)[:, None]
    hi = np.where(s[:, None] > 0, np.minimum(127, np.ceil(f32(top / d))), 0)
    lo = np.where(s[:, None] > 0, np.maximum(-127, np.floor(f32(low / d))), 0)
    return hi.astype(np.int8), lo.astype(np.int8), s.astype(np.float32)


def select(q, bounds, scales, table, lens, T, budget, sink, recent):
    """q [B, Hq, D], bounds int8 [P, H, 2, D]: index [B, H, budget], page table, lens, scores."""
    B, Hq, D = q.shape
    P, H = scales.shape
    G, maxp = Hq // H, table.shape[1]
    index = np.full((B, H, budget), -1, np.int64)
    out = np.full((B, H, budget), -1, np.int64)
    sel_lens = np.zeros((B, H), np.int64)
    scores = np.full((B, H, maxp), np.nan)
    for b in range(B):
        if lens[b] <= 0 or lens[b] > maxp * T:
            continue
        n = -(-int(lens[b]) // T)
        for h in range(H):
            sc = np.full(n, -np.inf)
            ids = table[b, :n]
            ok = (ids >= 0) & (ids < P)
            for g in range(G):
                x = np.asarray(q[b, h * G + g], dtype=np.float64)
                amax = np.abs(x).max() if np.isfinite(x).all() else 0.0
                f = f32(amax / 255)
                qi = np.rint(f32(x / f)) if f > 0 else np.zeros(D)
                box = bounds[np.where(ok, ids, 0), h].astype(np.float64)
                S = np.where(qi > 0, qi * box[:, 0], qi * box[:, 1]).sum(-1)
                sc = np.where(ok, np.maximum(sc, f32(f32(S * f) * scales[np.where(ok, ids, 0), h])), -np.inf)
            at = np.arange(n)
            forced = (at < sink) | (at >= n - recent)
            sc = np.where(forced, np.inf, sc)
            scores[b, h, :n] = sc
            order = sorted(range(n), key=lambda i: (not forced[i], -sc[i], i))[:budget]
            kept = np.array(sorted(order))
            index[b, h, :len(kept)] = kept
            out[b, h, :len(kept)] = ids[kept]
            sel_lens[b, h] = (len(kept) - 1) * T + int(lens[b]) - (n - 1) * T
    return index, out, sel_lens, scores


def attend(q, kd, ks, vd, vs, g_k, g_v, table, lens, T, sm_scale):
    """Attention of each (sequence, KV head) over its own pages: out [B, Hq, D], lse [B, Hq]."""
    B, Hq, D = q.shape
    H = kd.shape[1]
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    scale = f32(sm_scale) * float(g_k)
    for b in range(B):
        for h in range(H):
            n = int(lens[b, h])
            if n <= 0 or n > table.shape[2] * T:
                continue
            ids = table[b, h, :-(-n // T)]
            ok = (ids >= 0) & (ids < kd.shape[0])
            at = np.where(ok, ids, 0)
            k = keys(kd[at, h], ks[at, h]).reshape(-1, D)[:n]
            code = np.stack([vd[at, h] & 15, vd[at, h] >> 4], 2)            # [n, T/2, 2, D]
            sb = np.moveaxis(vs[at, h], -1, -2)                             # [n, T/2, 2, D/16]
            v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
            v = (v.reshape(*v.shape[:-1], -1, 16) * np.append(E4M3, 0.0)[sb & 127][..., None]).reshape(-1, D)[:n]
            here = np.repeat(ok, T)[:n]
            if not here.any():
                continue
            for g in range(h * G, (h + 1) * G):
                x = np.where(here, k @ np.asarray(q[b, g], dtype=np.float64) * scale, -np.inf)
                top = x.max()
                p = np.exp(x - top)
                lse[b, g] = top + np.log(p.sum())
                out[b, g] = p @ v * float(g_v) / p.sum()
    return out, lse
