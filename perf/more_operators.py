"""Cases of the operators around a cache of 8-bit pages and a sliding window: page tables and token slots of a step built
from request lengths, pages held as FP8 with a scale for each page and head, attention of single tokens and of chunks over
them, and the decode attention over NVFP4 pages with a sliding window and first tokens that stay visible.

`run` computes them in plain torch operations where `own` is false and through the library where it is true."""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a full batch: a token each, and some requests that ended: latency is everything
        _tables("tables, decode step of 256", 256, 64, 131072, 1, 1, done=0.05),
        # the chunks of an extend step: 16 sequences x 512 new tokens
        _tables("tables, 16 chunks of 512", 16, 64, 4096, 512, 512),
        # prompts of any length and decode tokens in one step, small pages, a pool that runs out
        _tables("tables, 700 ragged requests", 700, 16, 9000, 0, 150, done=0.1, short=True),
        # the pages of a prompt batch of 32 sequences x 8192 tokens
        _pages("fp8 pages, 4096 from bf16", 4096, 4096, 8, 128, 64),
        # the cached prefix of an extend step: 16 sequences x 4096 tokens out of the NVFP4 pool
        _pages("fp8 pages, 1024 from nvfp4", 1024, 1300, 8, 128, 64, src="nvfp4"),
        # a decode batch at 8192 tokens
        _decode("fp8 decode, batch of 32", 32, 32, 8, 128, 64, 8192, low=8192),
        # sequences of all lengths, some empty, wide heads, an odd group, small pages
        _decode("fp8 decode, ragged head 256", 19, 15, 5, 256, 16, 9000, window=2048, sinks=4),
        # long contexts of which a layer with a sliding window sees 4096 tokens and the first 4
        _window("window decode, batch of 32", 32, 32, 8, 128, 64, 131072, 4096, 4, low=32768),
        # a single user, head dim 64, a window that ends inside pages
        _window("window decode, one sequence", 1, 64, 8, 64, 16, 100003, 1000, 5, low=100003),
        # the chunks of an extend step behind their 4096-token prefixes
        _extend("extend, 16 chunks of 512", 16, 32, 8, 128, 64, 4096, 512, plow=4096, nlow=512),
        # one long prompt in chunks, late in the prompt
        _extend("extend, 2048 tokens at 65536", 1, 32, 8, 128, 64, 63488, 2048, plow=63488, nlow=2048),
        # prompts and decode tokens in one step, a sliding window, a group of 3, padding rows
        _extend("extend, ragged window head 64", 24, 12, 4, 64, 32, 1500, 700, window=600, sinks=4, padding=37),
    ]


def _tables(name, b, t, past, nlow, nhigh, done=0.0, short=False):
    return {"name": name, "op": "tables", "b": b, "t": t, "past": past, "nlow": nlow, "nhigh": nhigh, "done": done, "short": short}


def _pages(name, pages, pool, h, d, t, src="bf16", partial=False):
    return {"name": name, "op": "pages", "pages": pages, "pool": pool, "h": h, "d": d, "t": t, "src": src, "partial": partial}


def _decode(name, b, hq, h, d, t, high, low=0, window=0, sinks=0, blocks=True):
    return {"name": name, "op": "decode", "b": b, "hq": hq, "h": h, "d": d, "t": t, "low": low, "high": high, "window": window,
            "sinks": sinks, "blocks": blocks}


def _window(name, b, hq, h, d, t, high, window, sinks, low=0):
    return {"name": name, "op": "window", "b": b, "hq": hq, "h": h, "d": d, "t": t, "low": low, "high": high, "window": window, "sinks": sinks}


def _extend(name, b, hq, h, d, t, phigh, nhigh, plow=0, nlow=0, window=0, sinks=0, padding=0, blocks=True):
    return {"name": name, "op": "extend", "b": b, "hq": hq, "h": h, "d": d, "t": t, "plow": plow, "phigh": phigh, "nlow": nlow,
            "nhigh": nhigh, "window": window, "sinks": sinks, "padding": padding, "blocks": blocks}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "pages", "decode", "decode", "window", "window", "extend", "extend", "extend"))
    h, d, t = rng.randint(1, 8), rng.choice((64, 128, 256)), rng.choice((16, 32, 48, 64, 128))
    hq = h * rng.randint(1, 8)
    window, sinks = rng.choice((0, _log(rng, 1, 5000))), rng.choice((0, 1, 4, rng.randint(1, 100)))
    if op == "tables":
        b = _log(rng, 1, 1000)
        most = _log(rng, 1, max(1, min(2048, 100000 // b)))
        c = _tables("", b, t, _log(rng, 1, 131072), rng.choice((0, 1, most)), most, rng.choice((0.0, 0.1, 0.3)), rng.random() < 0.3)
    elif op == "pages":
        pages = _log(rng, 1, min(4096, 4096 * 8 * 128 * 64 // (h * d * t)))
        c = _pages("", pages, pages + rng.randint(0, 300), h, d, t, rng.choice(("bf16", "fp16", "nvfp4", "nvfp4 pairs")), rng.random() < 0.5)
    elif op == "decode":
        b = _log(rng, 1, 64)
        high = _log(rng, 1, max(1, min(131072, 32 * 8192 * 8 * 128 // (b * h * d))))
        c = _decode("", b, hq, h, d, t, high, rng.choice((0, high // 2, high)), window, sinks, rng.random() < 0.7)
    elif op == "window":
        b = _log(rng, 1, 64)
        high = _log(rng, 1, 131072)
        c = _window("", b, hq, h, d, t, high, max(1, min(window or 777, 32 * 4096 * 8 * 128 // (b * h * d))), sinks, rng.choice((0, high // 2, high)))
    else:
        b = _log(rng, 1, 32)
        rows = _log(rng, 1, max(1, 4096 // b))
        past = _log(rng, 1, max(1, min(32768, 2 ** 35 // (b * rows * hq * d), 16 * 8192 * 8 * 128 // (b * h * d))))
        c = _extend("", b, hq, h, d, t, past, rows, rng.choice((0, past)), rng.choice((0, 1, rows)), window, sinks, rng.choice((0, rng.randint(0, 50))),
                    rng.random() < 0.7)
    del c["name"]
    return c


def _pages_of(n, t):
    return (n + t - 1) // t


# ------------------------------------------------------------------------------------------ inputs

def _codes(shape, g, dev):
    return torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)


def _scales(shape, g, dev):
    """E4M3 bytes of 0.25 to 1."""
    return torch.randint(0x28, 0x39, shape, generator=g, device=dev, dtype=torch.uint8)


def _scalar(x, dev):
    return torch.tensor([x], dtype=torch.float32, device=dev)


def _between(low, high, n, g):
    """Lengths; where they start at 0, about one in eight is 0."""
    x = torch.randint(low, high + 1, (n,), generator=g)
    if low == 0:
        x[torch.rand(n, generator=g) < 0.125] = 0
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    cg, g = torch.Generator().manual_seed(seed), torch.Generator(device=dev).manual_seed(seed)
    return {"case": case, "e2m1": torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev), **_PREPARE[case["op"]](case, cg, g, dev)}


def _prepare_tables(c, cg, g, dev):
    b, t = c["b"], c["t"]
    past = _between(0, c["past"], b, cg)
    new = torch.randint(c["nlow"], c["nhigh"] + 1, (b,), generator=cg)
    new[torch.rand(b, generator=cg) < c["done"]] = -1
    have = _pages_of(past, t)
    need = torch.where(new > 0, _pages_of(past + new.clamp(min=0), t) - have, 0)
    maxp = _pages_of(c["past"] + c["nhigh"], t)
    used, back, want = int(have.sum()), int(have[new < 0].sum()), int(need.sum())
    free = max(0, want * 2 // 3 - back) if c["short"] else want + int(torch.randint(0, 100, (1,), generator=cg))
    perm = torch.randperm(used + free, generator=cg).to(torch.int32)
    first = have.cumsum(0) - have
    at = torch.arange(maxp)
    table = torch.where(at < have[:, None], perm[(first[:, None] + at).clamp(max=max(0, used + free - 1))] if used + free else 0, -1).to(torch.int32)
    stack = torch.full((b * maxp + 100,), -1, dtype=torch.int32)
    stack[:free] = perm[used:]
    rows = max(1, b * c["nhigh"])
    i32 = {"dtype": torch.int32, "device": dev}
    return {"past": past.to(torch.int32).to(dev), "new": new.to(torch.int32).to(dev), "table": table.to(dev), "stack": stack.to(dev),
            "count": torch.tensor([free], **i32), "left": torch.zeros(1, **i32), "lens": torch.zeros(b, **i32), "starts": torch.zeros(b + 1, **i32),
            "slots": torch.zeros(rows, dtype=torch.int64, device=dev), "positions": torch.zeros(rows, **i32),
            "full": torch.zeros(b + rows // t, **i32)}


def _prepare_pages(c, cg, g, dev):
    pages, pool, h, d, t = c["pages"], c["pool"], c["h"], c["d"], c["t"]
    s = {"from": torch.randperm(pool, generator=cg)[:pages].to(torch.int32).to(dev), "to": torch.randperm(pool, generator=cg)[:pages].to(torch.int32).to(dev),
         "tokens": torch.randint(0, t + 1, (pages,), generator=cg).to(torch.int32).to(dev) if c["partial"] else None,
         "dst": torch.zeros((pool, h, t, d), dtype=torch.float8_e4m3fn, device=dev), "dst_scales": torch.zeros((pool, h), device=dev)}
    if c["src"] in DTYPES:
        x = torch.randn((pool, h, t, d), generator=g, device=dev)
        x[..., [i for i in (13, 42, 77, 118) if i < d]] *= 20.0
        return {"src": x.to(DTYPES[c["src"]]), **s}
    pairs = c["src"] == "nvfp4 pairs"
    return {"src": _codes((pool, h, t // 2, d) if pairs else (pool, h, t, d // 2), g, dev),
            "src_scales": _scales((pool, h, t // 2, d // 16, 2) if pairs else (pool, h, t, d // 16), g, dev), "g": _scalar(0.03, dev), **s}


def _fp8_pool(c, pool, g, dev):
    """K and V pages as an encoder leaves them: the largest of a page and head near 448 steps of its scale."""
    h, d, t = c["h"], c["d"], c["t"]
    s = {}
    for x in "kv":
        s[x] = torch.randn((pool, h, t, d), generator=g, device=dev).mul_(112.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        s[x + "b"] = torch.rand((pool, h), generator=g, device=dev) * 0.008 + 0.005 if c["blocks"] else None
        s[x + "s"] = None if c["blocks"] else _scalar(0.009, dev)
    return s


def _table(n, maxp, first, cg, dev):
    """Page table of sequences that have pages first[i] .. n[i]; what they gave back is -1. And the pages of a pool."""
    have = torch.clamp(n - first, min=0)
    used = int(have.sum())
    pool = used + 7
    perm = torch.randperm(pool, generator=cg).to(torch.int32)
    at = torch.arange(maxp)
    start = have.cumsum(0) - have
    index = (start[:, None] + at - first[:, None]).clamp(0, pool - 1)
    return torch.where((at >= first[:, None]) & (at < n[:, None]), perm[index], -1).to(dev).contiguous(), pool


def _prepare_decode(c, cg, g, dev):
    b, hq, d, t = c["b"], c["hq"], c["d"], c["t"]
    lens = _between(c["low"], c["high"], b, cg)
    table, pool = _table(_pages_of(lens, t), max(1, _pages_of(c["high"], t)), torch.zeros_like(lens), cg, dev)
    return {"q": torch.randn((b, hq, d), generator=g, device=dev).to(torch.bfloat16), "table": table, "lens": lens.to(torch.int32).to(dev),
            "sm_scale": 1 / math.sqrt(d), "workspace": torch.empty(64 << 20, dtype=torch.uint8, device=dev),
            "out": torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev), "lse": torch.empty((b, hq), device=dev), **_fp8_pool(c, pool, g, dev)}


def _prepare_window(c, cg, g, dev):
    b, hq, h, d, t = c["b"], c["hq"], c["h"], c["d"], c["t"]
    lens = _between(c["low"], c["high"], b, cg)
    n, maxp = _pages_of(lens, t), max(1, _pages_of(c["high"], t))
    # the pages between the first tokens and the window have been given back
    first = (lens - c["window"]).clamp(min=0) // t
    keep = torch.minimum(first, torch.tensor(_pages_of(c["sinks"], t)))
    held = n - first + keep
    pool = int(held.sum()) + 7
    perm = torch.randperm(pool, generator=cg).to(torch.int32)
    at = torch.arange(maxp)
    start = (held.cumsum(0) - held)[:, None]
    index = torch.where(at < keep[:, None], at, at - (first - keep)[:, None]) + start
    here = (at < keep[:, None]) | ((at >= first[:, None]) & (at < n[:, None]))
    table = torch.where(here, perm[index.clamp(0, pool - 1)], -1)
    return {"q": torch.randn((b, hq, d), generator=g, device=dev).to(torch.bfloat16), "table": table.to(dev).contiguous(), "lens": lens.to(torch.int32).to(dev),
            "kd": _codes((pool, h, t, d // 2), g, dev), "ks": _scales((pool, h, t, d // 16), g, dev),
            "vd": _codes((pool, h, t // 2, d), g, dev), "vs": _scales((pool, h, t // 2, d // 16, 2), g, dev), "gk": _scalar(1.0, dev), "gv": _scalar(0.7, dev),
            "sm_scale": 1 / math.sqrt(d), "workspace": torch.empty(64 << 20, dtype=torch.uint8, device=dev),
            "out": torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev), "lse": torch.empty((b, hq), device=dev)}


def _prepare_extend(c, cg, g, dev):
    b, hq, d, t = c["b"], c["hq"], c["d"], c["t"]
    past, new = _between(c["plow"], c["phigh"], b, cg), _between(c["nlow"], c["nhigh"], b, cg)
    lens = past + new
    table, pool = _table(_pages_of(lens, t), max(1, _pages_of(c["phigh"] + c["nhigh"], t)), torch.zeros_like(lens), cg, dev)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    rows = b * c["nhigh"] + c["padding"]  # of a captured step: those that a step does not fill are padding
    return {"q": torch.randn((rows, hq, d), generator=g, device=dev).to(torch.bfloat16), "table": table, "lens": lens.to(torch.int32).to(dev),
            "starts": starts.to(torch.int32).to(dev), "sm_scale": 1 / math.sqrt(d), "workspace": torch.empty(256 << 20, dtype=torch.uint8, device=dev),
            "out": torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=dev), "lse": torch.zeros((rows, hq), device=dev), **_fp8_pool(c, pool, g, dev)}


_PREPARE = {"tables": _prepare_tables, "pages": _prepare_pages, "decode": _prepare_decode, "window": _prepare_window, "extend": _prepare_extend}


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _tables_outputs(s):
    return {x: s[x] for x in ("lens", "starts", "slots", "positions", "full", "left", "table", "stack")}


def _own_tables(s):
    import nvfp4_paged_kv_gb300 as kv
    kv.nvfp4_kv_step_tables(kv.Layout(1, 64, s["case"]["t"]), s["past"], s["new"], s["stack"], s["count"], s["table"], s["lens"], s["starts"], s["slots"],
                            s["positions"], free_left=s["left"], full_pages=s["full"])
    return _tables_outputs(s)


def _own_pages(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    layout = kv.Layout(c["h"], c["d"], c["t"], kv.PACK_TOKEN_PAIRS if c["src"] == "nvfp4 pairs" else kv.PACK_DIM_PAIRS)
    kv.nvfp4_kv_fp8_pages(layout, s["src"], s["dst"], s["dst_scales"], src_scales=s.get("src_scales"), global_scale=s.get("g"), src_page_ids=s["from"],
                          dst_page_ids=s["to"], page_tokens=s["tokens"])
    return {"values": s["dst"], "scales": s["dst_scales"]}


def _own_decode(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_paged_fp8_decode_attention(kv.Layout(c["h"], c["d"], c["t"]), s["q"], s["k"], s["v"], s["table"], s["lens"], s["sm_scale"], s["out"],
                                        k_block_scales=s["kb"], v_block_scales=s["vb"], k_scale=s["ks"], v_scale=s["vs"], window=c["window"],
                                        sink_tokens=c["sinks"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_window(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_paged_window_decode_attention(kv.Layout(c["h"], c["d"], c["t"]), s["q"], s["kd"], s["ks"], s["gk"], s["vd"], s["vs"], s["gv"], s["table"],
                                           s["lens"], s["sm_scale"], s["out"], window=c["window"], sink_tokens=c["sinks"], lse=s["lse"],
                                           workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_extend(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_paged_extend_attention(kv.Layout(c["h"], c["d"], c["t"]), s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], s["sm_scale"], s["out"],
                                    k_block_scales=s["kb"], v_block_scales=s["vb"], k_scale=s["ks"], v_scale=s["vs"], window=c["window"],
                                    sink_tokens=c["sinks"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tables(s):
    t, maxp, cap, rows = s["case"]["t"], s["table"].shape[1], s["stack"].shape[0], s["slots"].shape[0]
    past, new = s["past"].long(), s["new"].long()
    dev, b = past.device, past.shape[0]
    have = _pages_of(past, t)
    # pages of requests that ended go on the stack, in order
    back = torch.where(new < 0, have, 0)
    ends = back.cumsum(0)
    i = torch.arange(cap, device=dev)
    who = torch.searchsorted(ends, i - s["count"], right=True).clamp(max=b - 1)
    page = (i - s["count"] - (ends - back)[who]).clamp(0, maxp - 1)
    pushed = (i >= s["count"]) & (i < s["count"] + ends[-1])
    stack = torch.where(pushed, s["table"][who, page], s["stack"])
    top = s["count"] + ends[-1]
    # pages are dealt from its top, to the requests in order
    add = new.clamp(min=0)
    need = torch.where(add > 0, _pages_of(past + add, t) - have, 0)
    upto = need.cumsum(0)
    served = (new >= 0) & ((need == 0) | (upto <= top))
    lens = torch.where(new < 0, 0, torch.where(served, past + add, past))
    at = torch.arange(maxp, device=dev)
    k = (upto - need)[:, None] + at - have[:, None]
    fresh = served[:, None] & (at >= have[:, None]) & (at < (have + need)[:, None])
    table = torch.where(fresh, stack[(top - 1 - k).clamp(0, cap - 1)], s["table"])
    # rows of the step
    starts = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0)])
    r = torch.arange(rows, device=dev)
    who = (torch.searchsorted(starts, r, right=True) - 1).clamp(max=b - 1)
    pos = past[who] + r - starts[who]
    real = r < starts[-1]
    good = real & served[who]
    slots = torch.where(good, table[who, torch.where(good, pos // t, 0)].long() * t + pos % t, -1)
    # pages that became full
    full = torch.where(served, (past + add) // t - past // t, 0)
    fends = full.cumsum(0)
    i = torch.arange(s["full"].shape[0], device=dev)
    who = torch.searchsorted(fends, i, right=True).clamp(max=b - 1)
    page = (past // t)[who] + i - (fends - full)[who]
    s["full"].copy_(torch.where(i < fends[-1], table[who, page.clamp(0, maxp - 1)], -1))
    s["slots"].copy_(slots)
    s["positions"].copy_(torch.where(good, pos, 0))
    s["lens"].copy_(lens)
    s["starts"].copy_(starts)
    s["left"].copy_(top - torch.where(served, need, 0).sum())
    s["table"].copy_(table)
    s["stack"].copy_(stack)
    return _tables_outputs(s)


def _keys(data, scales, e2m1):
    """Values without the tensor's scale: codes [.., t, d / 2] and scale bytes [.., t, d / 16] to [.., t, d]."""
    x = e2m1[torch.stack([data & 15, data >> 4], -1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _values(data, scales, e2m1):
    """The same of codes [.., t / 2, d] and scale bytes [.., t / 2, d / 16, 2]."""
    x = e2m1[torch.stack([data & 15, data >> 4], -2).int()]
    sc = scales.view(torch.float8_e4m3fn).float().movedim(-1, -2)
    return (x.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2).flatten(-3, -2)


def _plain_pages(s):
    c = s["case"]
    src, to = s["from"].long(), s["to"].long()
    if c["src"] in DTYPES:
        x = s["src"][src].float()
    else:
        x = (_values if c["src"] == "nvfp4 pairs" else _keys)(s["src"][src], s["src_scales"][src], s["e2m1"]) * s["g"]
    if s["tokens"] is not None:
        x = torch.where((torch.arange(c["t"], device=x.device) < s["tokens"][:, None])[:, None, :, None], x, 0.0)
    # (a number as the divisor would be turned into a product with its reciprocal)
    top = x.abs().amax((2, 3))
    scale = top / torch.full_like(top[:1, :1], 448)
    scale = torch.where(scale < 2.0 ** -100, 1.0, scale)
    s["dst"][to] = (x * (1.0 / scale)[..., None, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    s["dst_scales"][to] = scale
    return {"values": s["dst"], "scales": s["dst_scales"]}


def _attention(q, k, v, pos, at, there, window, sinks):
    """q [.., rows, d], k and v [.., tokens, d] of positions `at` [.., tokens], rows at positions pos [.., rows]: out and lse."""
    x = torch.matmul(q, k.transpose(-1, -2))
    pos, at = pos[..., None], at[..., None, :]
    here = there[..., None, :] & (at <= pos)
    if window:
        here = here & ((at > pos - window) | (at < sinks))
    x = torch.where(here, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    p = torch.exp(x - torch.where(some, top, 0.0))
    del x, here
    total = p.sum(-1, keepdim=True)
    out = torch.where(some, torch.matmul(p, v) / total, 0.0)
    return out, torch.where(some, top + torch.log(total), -math.inf)[..., 0]


def _fp8_tokens(s, x):
    """K or V [b, h, tokens, d] of the page table in 32 bits."""
    ids = s["table"].long().clamp(min=0)
    y = s[x][ids].float()
    y = y * (s[x + "b"][ids][..., None, None] if s[x + "b"] is not None else s[x + "s"])
    return y.transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    b, h, d = c["b"], c["h"], c["d"]
    k, v = _fp8_tokens(s, "k"), _fp8_tokens(s, "v")
    at = torch.arange(k.shape[2], device=k.device)[None, None]
    lens = s["lens"].long()[:, None, None]
    out, lse = _attention(s["q"].float().view(b, h, -1, d) * s["sm_scale"], k, v, lens - 1, at, at < lens, c["window"], c["sinks"])
    s["out"].copy_(out.reshape(b, -1, d))
    s["lse"].copy_(lse.reshape(b, -1))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_window(s):
    c = s["case"]
    b, h, d, t, maxp = c["b"], c["h"], c["d"], c["t"], s["table"].shape[1]
    lens = s["lens"].long()
    first = (lens - c["window"]).clamp(min=0) // t
    keep, count = _pages_of(c["sinks"], t), _pages_of(c["window"], t) + 1
    dev = lens.device
    # the first pages, then those of the window; a page that is among both counts once
    page = torch.cat([torch.arange(keep, device=dev).expand(b, keep), first[:, None] + torch.arange(count, device=dev)], 1)
    there = torch.cat([torch.arange(keep, device=dev) < first[:, None], (first[:, None] + torch.arange(count, device=dev)) * t < lens[:, None]], 1)
    ids = s["table"].long().gather(1, page.clamp(max=maxp - 1)).clamp(min=0)
    at = (page[..., None] * t + torch.arange(t, device=dev)).flatten(1)
    there = there.repeat_interleave(t, 1) & (at < lens[:, None])
    k = _keys(s["kd"][ids], s["ks"][ids], s["e2m1"]).transpose(1, 2).flatten(2, 3) * s["gk"]
    v = _values(s["vd"][ids], s["vs"][ids], s["e2m1"]).transpose(1, 2).flatten(2, 3) * s["gv"]
    out, lse = _attention(s["q"].float().view(b, h, -1, d) * s["sm_scale"], k, v, (lens - 1)[:, None, None], at[:, None], there[:, None], c["window"],
                          c["sinks"])
    s["out"].copy_(out.reshape(b, -1, d))
    s["lse"].copy_(lse.reshape(b, -1))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_extend(s):
    c = s["case"]
    b, hq, h, d, most = c["b"], c["hq"], c["h"], c["d"], c["nhigh"]
    rows, dev = s["q"].shape[0], s["q"].device
    starts, lens = s["starts"].long(), s["lens"].long()
    i = torch.arange(most, device=dev)
    row = (starts[:-1, None] + i).clamp(max=rows - 1)
    new = starts[1:] - starts[:-1]
    # [b, h, group x rows, d]: rows of a sequence side by side, padded to the longest
    q = (s["q"][row].float() * s["sm_scale"]).view(b, most, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    pos = ((lens - new)[:, None] + i)[:, None, None].expand(b, 1, hq // h, most).reshape(b, 1, -1)
    k, v = _fp8_tokens(s, "k"), _fp8_tokens(s, "v")
    at = torch.arange(k.shape[2], device=dev)[None, None]
    out, lse = _attention(q, k, v, pos, at, at < lens[:, None, None], c["window"], c["sinks"])
    out = out.view(b, hq, most, d).transpose(1, 2)
    lse = lse.view(b, hq, most).transpose(1, 2)
    r = torch.arange(rows, device=dev)
    who = (torch.searchsorted(starts, r, right=True) - 1).clamp(max=b - 1)
    nth = (r - starts[who]).clamp(max=most - 1)
    real = r < starts[-1]
    s["out"].copy_(torch.where(real[:, None, None], out[who, nth], s["out"].float()))
    s["lse"].copy_(torch.where(real[:, None], lse[who, nth], s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


_OWN = {"tables": _own_tables, "pages": _own_pages, "decode": _own_decode, "window": _own_window, "extend": _own_extend}
_PLAIN = {"tables": _plain_tables, "pages": _plain_pages, "decode": _plain_decode, "window": _plain_window, "extend": _plain_extend}


# ------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    return _WORK[case["op"]](case)


def _work_tables(c):
    b, rows = c["b"], c["b"] * c["nhigh"]
    new = b * (c["nlow"] + c["nhigh"]) / 2
    pages = new / c["t"] + (c["done"] * b * c["past"] / 2 / c["t"])
    return {"bytes": rows * 12 + b * 20 + pages * 8 + (b + rows // c["t"]) * 4, "flops": rows * 4 + b * 10}


def _work_pages(c):
    values = c["pages"] * c["h"] * c["t"] * c["d"]
    real = values * (0.5 if c["partial"] else 1.0)
    return {"bytes": real * (2 if c["src"] in DTYPES else 9 / 16) + values + c["pages"] * (c["h"] * 4 + 8), "flops": real * 3}


def _seen(pos, window, sinks):
    """Tokens that a row at this position sees."""
    return pos + 1 if not window else min(pos + 1, window + sinks)


def _work_decode(c):
    tokens = c["b"] * _seen((c["low"] + c["high"]) / 2 - 1, c["window"], c["sinks"])
    return {"bytes": tokens * c["h"] * c["d"] * 2 + c["b"] * c["hq"] * (c["d"] * 4 + 4), "flops": tokens * c["hq"] * c["d"] * 4}


def _work_window(c):
    tokens = c["b"] * _seen((c["low"] + c["high"]) / 2 - 1, c["window"], c["sinks"])
    return {"bytes": tokens * c["h"] * c["d"] * 9 / 8 + c["b"] * c["hq"] * (c["d"] * 4 + 4), "flops": tokens * c["hq"] * c["d"] * 4}


def _work_extend(c):
    past, new = (c["plow"] + c["phigh"]) / 2, (c["nlow"] + c["nhigh"]) / 2
    if c["window"]:
        full = max(0.0, min(new, past + new - (c["window"] + c["sinks"])))  # rows whose window is full
        part = new - full
        pairs = full * (c["window"] + c["sinks"]) + part * (past + part / 2)
        tokens = min(past + new, c["window"] + c["sinks"] + new)
    else:
        pairs, tokens = new * (past + new / 2), past + new
    return {"bytes": c["b"] * (tokens * c["h"] * c["d"] * 2 + new * c["hq"] * (c["d"] * 4 + 4)), "flops": max(1.0, c["b"] * pairs * c["hq"] * c["d"] * 4)}


_WORK = {"tables": _work_tables, "pages": _work_pages, "decode": _work_decode, "window": _work_window, "extend": _work_extend}


# ------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["op"] == "tables":  # whole numbers
        return None
    return _EXACT[case["op"]](prepare(case, seed))


def _grid(x, e2m1):
    return e2m1.double()[x.long()]


def _unpacked(codes, scales, pairs, e2m1):
    """NVFP4 pages [n, t, d] of one head or of all, in 64 bits."""
    if pairs:
        x = torch.empty((*codes.shape[:-2], codes.shape[-2] * 2, codes.shape[-1]), dtype=torch.float64, device=codes.device)
        x[..., 0::2, :], x[..., 1::2, :] = _grid(codes & 15, e2m1), _grid(codes >> 4, e2m1)
        sc = scales.view(torch.float8_e4m3fn).double()
        each = torch.empty((*x.shape[:-1], x.shape[-1] // 16), dtype=torch.float64, device=codes.device)
        each[..., 0::2, :], each[..., 1::2, :] = sc[..., 0], sc[..., 1]
    else:
        x = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=codes.device)
        x[..., 0::2], x[..., 1::2] = _grid(codes & 15, e2m1), _grid(codes >> 4, e2m1)
        each = scales.view(torch.float8_e4m3fn).double()
    return x * each.repeat_interleave(16, -1)


def _exact_pages(s):
    """The scales: the largest magnitude among the page's tokens over 448, or 1."""
    c, scales = s["case"], s["dst_scales"].double().clone()
    for i in torch.arange(c["pages"], device=scales.device).split(256):
        src = s["from"][i].long()
        if c["src"] in DTYPES:
            x = s["src"][src].double()
        else:
            x = _unpacked(s["src"][src], s["src_scales"][src], c["src"] == "nvfp4 pairs", s["e2m1"]) * s["g"].double()
        if s["tokens"] is not None:
            x[(torch.arange(c["t"], device=x.device) >= s["tokens"][i][:, None])[:, None].expand(x.shape[:3])] = 0.0
        top = x.abs().flatten(2).amax(-1) / 448
        scales[s["to"][i].long()] = torch.where(top < 2.0 ** -100, 1.0, top)
    return {"values": None, "scales": scales}


def _exact_rows(q, k, v, pos, at, c, scale):
    """Rows [n, d] at positions pos [n] over tokens at positions `at`, a few rows at a time."""
    out, lse = [], []
    for qs, ps in zip(q.split(2048), pos.split(2048)):
        x = qs.double() @ k.t() * scale
        hide = at > ps[:, None]
        if c["window"]:
            hide |= (at <= ps[:, None] - c["window"]) & (at >= c["sinks"])
        x[hide] = -math.inf
        lse.append(torch.logsumexp(x, -1))
        out.append(torch.exp(x - lse[-1][:, None]) @ v)
    return torch.cat(out), torch.cat(lse)


def _sm_scale(s):
    return float(torch.tensor(s["sm_scale"], dtype=torch.float32))


def _fp8_head(s, x, ids, j, n):
    y = s[x][ids, j].double()
    y = y * (s[x + "b"][ids, j].double()[:, None, None] if s[x + "b"] is not None else s[x + "s"].double())
    return y.reshape(-1, y.shape[-1])[:n]


def _exact_attention(s, out, lse, rows, heads):
    """rows: for each sequence the rows of q, out and lse and their positions; heads(i, j): its tokens' k, v and positions."""
    c = s["case"]
    group = c["hq"] // c["h"]
    for i, (where, pos) in enumerate(rows):
        if not len(pos):
            continue
        for j in range(c["h"]):
            k, v, at = heads(i, j)
            if not len(at):
                out[where, j * group:(j + 1) * group], lse[where, j * group:(j + 1) * group] = 0.0, -math.inf
                continue
            q = s["q"][where, j * group:(j + 1) * group]
            o, m = _exact_rows(q.reshape(-1, c["d"]), k, v, pos.repeat_interleave(group), at, c, _sm_scale(s))
            out[where, j * group:(j + 1) * group], lse[where, j * group:(j + 1) * group] = o.view(q.shape), m.view(q.shape[:2])
    return {"out": out, "lse": lse}


def _exact_decode(s):
    c, lens, dev = s["case"], s["lens"].tolist(), s["q"].device
    rows = [(slice(i, i + 1), torch.tensor([n - 1], device=dev)) for i, n in enumerate(lens)]

    def heads(i, j):
        ids = s["table"][i, :_pages_of(lens[i], c["t"])].long()
        return _fp8_head(s, "k", ids, j, lens[i]), _fp8_head(s, "v", ids, j, lens[i]), torch.arange(lens[i], device=dev)

    return _exact_attention(s, torch.zeros_like(s["q"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64), rows, heads)


def _exact_window(s):
    c, lens, dev = s["case"], s["lens"].tolist(), s["q"].device
    rows = [(slice(i, i + 1), torch.tensor([n - 1], device=dev)) for i, n in enumerate(lens)]

    def heads(i, j):
        at = torch.arange(lens[i], device=dev)
        at = at[(at >= lens[i] - c["window"]) | (at < c["sinks"])]
        page, where = torch.unique(at // c["t"], return_inverse=True)
        ids = s["table"][i].long()[page]
        k = _unpacked(s["kd"][ids, j], s["ks"][ids, j], False, s["e2m1"]) * s["gk"].double()
        v = _unpacked(s["vd"][ids, j], s["vs"][ids, j], True, s["e2m1"]) * s["gv"].double()
        return k[where, at % c["t"]], v[where, at % c["t"]], at

    return _exact_attention(s, torch.zeros_like(s["q"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64), rows, heads)


def _exact_extend(s):
    c, lens, starts, dev = s["case"], s["lens"].tolist(), s["starts"].tolist(), s["q"].device
    if work(c)["flops"] > 6e12:
        return None
    rows = [(slice(a, e), torch.arange(n - (e - a), n, device=dev)) for a, e, n in zip(starts, starts[1:], lens)]

    def heads(i, j):
        ids = s["table"][i, :_pages_of(lens[i], c["t"])].long()
        return _fp8_head(s, "k", ids, j, lens[i]), _fp8_head(s, "v", ids, j, lens[i]), torch.arange(lens[i], device=dev)

    return _exact_attention(s, s["out"].double(), s["lse"].double(), rows, heads)


_EXACT = {"pages": _exact_pages, "decode": _exact_decode, "window": _exact_window, "extend": _exact_extend}
