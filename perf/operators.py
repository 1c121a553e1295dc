"""Cases of the cache operators of a decode step: appending a step's rows to the NVFP4 cache with the position
rotation, the bounds of a page's keys, the selection of pages by those bounds, and attention over the selected pages.

`run` computes them in plain torch operations where `own` is false and through the library where it is true."""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: each sequence adds one token; latency is everything
        _append("append, decode step of 32", 32, 32, 32, 8, 128, 64),
        # the chunk of an extend step: 16 sequences x 512 new tokens, starting anywhere in a page
        _append("append, 16 chunks of 512", 8192, 16, 32, 8, 128, 64),
        # ragged chunks and padding rows, FP16, adjacent pairs rotated in a part of the head, small pages
        _append("append, ragged fp16 head 256", 1237, 5, 20, 4, 256, 16, dtype="fp16", style="pairs", first=192, dims=64, padding=3),
        # after a prefill: the pages of 32 sequences x 8192 tokens
        _bounds("bounds, 4096 pages", 4096, 4096, 8, 128, 64),
        # pages that became full in one decode step, and ones cut short, out of a large pool
        _bounds("bounds, 37 partial pages", 37, 1000, 4, 64, 48, partial=True),
        # eight long contexts, 64 query and 8 KV heads
        _select("select, 8 long contexts", 8, 64, 8, 128, 64, 131072, 128, low=32768),
        # a decode batch at 8192 tokens: most of the cost is latency
        _select("select, batch of 32", 32, 32, 8, 128, 64, 8192, 32, low=8192),
        # one long prompt in small pages, few heads: little parallel work
        _select("select, one sequence page 16", 1, 6, 2, 64, 16, 100003, 200, low=100003),
        # eight long contexts, 8192 tokens kept of each
        _attend("attend, 8 long contexts", 8, 64, 8, 128, 64, 131072, 128, low=32768),
        # a decode batch, 2048 tokens kept of each sequence
        _attend("attend, batch of 32", 32, 32, 8, 128, 64, 8192, 32, low=8192),
        # a single user
        _attend("attend, one sequence", 1, 32, 8, 128, 64, 131072, 64, low=131072),
        # short and empty sequences among longer ones, small pages, wide heads, an odd group
        _attend("attend, ragged head 256", 19, 15, 5, 256, 16, 9000, 150),
    ]


def _append(name, rows, seqs, hq, h, d, t, dtype="bf16", style="halves", first=0, dims=0, padding=0):
    return {"name": name, "op": "append", "rows": rows, "seqs": seqs, "hq": hq, "h": h, "d": d, "t": t, "dtype": dtype,
            "style": style, "first": first, "dims": dims or d, "padding": padding}


def _bounds(name, pages, pool, h, d, t, partial=False):
    return {"name": name, "op": "bounds", "pages": pages, "pool": pool, "h": h, "d": d, "t": t, "partial": partial}


def _select(name, b, hq, h, d, t, high, budget, low=0, sink=1, recent=2):
    return {"name": name, "op": "select", "b": b, "hq": hq, "h": h, "d": d, "t": t, "low": low, "high": high,
            "budget": budget, "sink": sink, "recent": recent}


def _attend(name, b, hq, h, d, t, high, budget, low=0):
    return {"name": name, "op": "attend", "b": b, "hq": hq, "h": h, "d": d, "t": t, "low": low, "high": high, "budget": budget}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "bounds", "select", "attend", "attend"))
    h, d, t = rng.randint(1, 8), rng.choice((64, 128, 256)), rng.choice((16, 32, 48, 64, 128))
    hq = h * rng.randint(1, 8)
    if op == "append":
        rows = _log(rng, 1, min(8192, 8192 * 48 * 128 // ((hq + 2 * h) * d)))
        style = rng.choice(("halves", "pairs", "none"))
        dims = rng.choice([x for x in (32, 64, 128, 256) if x <= d])
        first = rng.choice((0, d - dims)) if style != "none" else 0
        c = _append("", rows, rng.randint(1, min(rows, 40)), hq, h, d, t, rng.choice(("bf16", "fp16")), style, first, dims,
                    rng.choice((0, 0, rng.randint(0, rows // 3))))
    elif op == "bounds":
        pages = _log(rng, 1, min(4096, 4096 * 8 * 128 * 64 // (h * d * t)))
        c = _bounds("", pages, pages + rng.randint(0, 500), h, d, t, rng.random() < 0.5)
    elif op == "select":
        b = _log(rng, 1, 48)
        high = _log(rng, 1, max(1, min(131072, 8 * 131072 * 8 * 128 // (b * h * d) * t // 64)))
        budget = _log(rng, 1, 300)
        sink = rng.randint(0, min(4, budget - 1))
        c = _select("", b, hq, h, d, t, high, budget, rng.choice((0, high // 2)), sink, rng.randint(1, min(4, budget - sink)))
    else:
        b = _log(rng, 1, 64)
        budget = _log(rng, 1, max(1, min(300, 8 * 8 * 8192 * 128 // (b * h * d * t))))
        c = _attend("", b, hq, h, d, t, _log(rng, 1, 131072), budget, 0)
        c["low"] = rng.choice((0, c["high"] // 2, c["high"]))
    del c["name"]
    return c


def _lens(c, g):
    """Lengths of a case's sequences; where they start at 0, about one in eight is empty."""
    n = torch.randint(c["low"], c["high"] + 1, (c["b"],), generator=g)
    if c["low"] == 0:
        n[torch.rand(c["b"], generator=g) < 0.125] = 0
    return n


def _pages(n, t):
    return (n + t - 1) // t


# ------------------------------------------------------------------------------------------ inputs

def _codes(shape, g, dev):
    return torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)


def _scales(shape, g, dev):
    """E4M3 bytes of 0.25 to 1."""
    return torch.randint(0x28, 0x39, shape, generator=g, device=dev, dtype=torch.uint8)


def _pool(pages, h, t, d, g, dev):
    """K codes and scales (two dims of a token in a byte), V codes and scales (two tokens of a dim in a byte)."""
    return {"kd": _codes((pages, h, t, d // 2), g, dev), "ks": _scales((pages, h, t, d // 16), g, dev),
            "vd": _codes((pages, h, t // 2, d), g, dev), "vs": _scales((pages, h, t // 2, d // 16, 2), g, dev)}


def _scalar(x, dev):
    return torch.tensor([x], dtype=torch.float32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    cg, g = torch.Generator().manual_seed(seed), torch.Generator(device=dev).manual_seed(seed)
    return {"case": case, "e2m1": torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev), **_PREPARE[case["op"]](case, cg, g, dev)}


def _prepare_append(c, cg, g, dev):
    rows, seqs, hq, h, d, t, dt = c["rows"], c["seqs"], c["hq"], c["h"], c["d"], c["t"], DTYPES[c["dtype"]]
    real = rows - c["padding"]
    cut = torch.sort(torch.randint(0, real + 1, (seqs - 1,), generator=cg)).values.tolist() if seqs > 1 else []
    if rows % seqs == 0 and not c["padding"]:
        cut = [rows // seqs * i for i in range(1, seqs)]
    ends = cut + [real]
    far = 32768
    slots, positions, page, need = [], [], 0, []
    for i, e in enumerate(ends):
        n = e - ([0] + ends)[i]
        start = int(torch.randint(0, far - n, (1,), generator=cg))
        need.append((start, n, page))
        page += _pages(torch.tensor(start % t + n), t).item()
    pool = _pages(torch.tensor(real), t).item() + 2 * seqs + 8
    assert page <= pool
    perm = torch.randperm(pool, generator=cg)
    for start, n, p in need:
        at = start + torch.arange(n)
        slots.append(perm[p + at // t - start // t] * t + at % t)
        positions.append(at)
    pad = torch.full((c["padding"],), -1)
    slots = torch.cat(slots + [pad])
    qkv = torch.randn((rows, (hq + 2 * h) * d), generator=g, device=dev)
    qkv[:, hq * d:(hq + h) * d].view(rows, h, d)[:, :, [x for x in (13, 42, 77, 118) if x < d]] *= 20.0
    qkv = qkv.to(dt)
    angle = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
        -torch.arange(0, c["dims"], 2, dtype=torch.float64, device=dev) / c["dims"])
    good = slots >= 0
    whole = torch.arange(rows)
    return {
        "q": qkv[:, :hq * d].view(rows, hq, d), "k": qkv[:, hq * d:(hq + h) * d].view(rows, h, d), "v": qkv[:, (hq + h) * d:].view(rows, h, d),
        "slots": slots.to(dev), "positions": torch.cat(positions + [torch.zeros_like(pad)]).to(torch.int32).to(dev),
        "table": torch.cat([angle.cos(), angle.sin()], 1).float(), "gk": _scalar(0.03, dev), "gv": _scalar(0.002, dev),
        "q_out": torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=dev),
        "k_out": torch.zeros((rows, h, d), dtype=torch.bfloat16, device=dev), "v_out": torch.zeros((rows, h, d), dtype=torch.bfloat16, device=dev),
        # the scheduler that made the slots knows which rows are real and which tokens are the first and second of a pair
        "real": whole[good].to(dev), "even": whole[good & (slots % 2 == 0)].to(dev), "odd": whole[good & (slots % 2 == 1)].to(dev),
        **_pool(pool, h, t, d, g, dev),
    }


def _prepare_bounds(c, cg, g, dev):
    pages, pool, h, d, t = c["pages"], c["pool"], c["h"], c["d"], c["t"]
    tokens = torch.randint(0, t + 1, (pages,), generator=cg) if c["partial"] else torch.full((pages,), t)
    return {"kd": _codes((pool, h, t, d // 2), g, dev), "ks": _scales((pool, h, t, d // 16), g, dev),
            "pages": torch.randperm(pool, generator=cg)[:pages].to(torch.int32).to(dev), "tokens": tokens.to(torch.int32).to(dev),
            "bounds": torch.zeros((pool, h, 2, d), dtype=torch.int8, device=dev), "bound_scales": torch.zeros((pool, h), device=dev)}


def _prepare_select(c, cg, g, dev):
    b, hq, h, d, t = c["b"], c["hq"], c["h"], c["d"], c["t"]
    lens = _lens(c, cg)
    n = _pages(lens, t)
    maxp, pool = max(1, int(_pages(torch.tensor(c["high"]), t))), int(n.sum()) + 7
    perm, table, at = torch.randperm(pool, generator=cg), torch.zeros((b, maxp), dtype=torch.int32), 0
    for i in range(b):
        table[i, :n[i]] = perm[at:at + int(n[i])].to(torch.int32)
        at += int(n[i])
    # a page's keys spread around a centre that differs from page to page, in units of 1/127 of the largest
    mid = torch.randn((pool, h, 1, d), generator=g, device=dev) * 12
    wide = torch.rand((pool, h, 1, d), generator=g, device=dev) * 60 + 10
    bounds = torch.cat([mid + wide, mid - wide], 2).round().clamp(-127, 127).to(torch.int8)
    return {"q": torch.randn((b, hq, d), generator=g, device=dev).to(torch.bfloat16), "bounds": bounds,
            "bound_scales": torch.rand((pool, h), generator=g, device=dev) * 0.02 + 0.04, "page_table": table.to(dev),
            "lens": lens.to(torch.int32).to(dev), "sel_table": torch.empty((b, h, c["budget"]), dtype=torch.int32, device=dev),
            "sel_index": torch.empty((b, h, c["budget"]), dtype=torch.int32, device=dev),
            "sel_lens": torch.empty((b, h), dtype=torch.int32, device=dev), "scores": torch.zeros((b, h, maxp), device=dev)}


def _prepare_attend(c, cg, g, dev):
    b, hq, h, d, t, budget = c["b"], c["hq"], c["h"], c["d"], c["t"], c["budget"]
    lens = _lens(c, cg)
    count = _pages(lens, t).clamp(max=budget)
    tokens = torch.where(count > 0, (count - 1) * t + (lens - 1) % t + 1, count)
    # every head of a sequence keeps pages of its own, out of the few more that its sequence is given in this pool
    each = max(1, int(_pages(torch.tensor(c["high"]), t).clamp(max=budget + budget // 2 + 1)))
    pool = b * each
    table = torch.rand((b, h, each), generator=cg).argsort(-1)[:, :, :budget].sort(-1).values
    table = torch.randperm(pool, generator=cg).view(b, 1, each).expand(b, h, each).gather(2, table)
    table = torch.cat([table, torch.zeros((b, h, budget - table.shape[2]), dtype=torch.int64)], 2)
    table = torch.where(torch.arange(budget) < count[:, None, None], table, -1)
    return {"q": torch.randn((b, hq, d), generator=g, device=dev).to(torch.bfloat16), "gk": _scalar(1.0, dev), "gv": _scalar(0.7, dev),
            "sel_table": table.to(torch.int32).to(dev).contiguous(), "sel_lens": tokens[:, None].expand(b, h).to(torch.int32).to(dev).contiguous(),
            "sm_scale": 1 / math.sqrt(d), "workspace": torch.empty(32 << 20, dtype=torch.uint8, device=dev), "out": torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev),
            "lse": torch.empty((b, hq), device=dev), **_pool(pool, h, t, d, g, dev)}


_PREPARE = {"append": _prepare_append, "bounds": _prepare_bounds, "select": _prepare_select, "attend": _prepare_attend}


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_append(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    rotary = None
    if c["style"] != "none":
        rotary = kv.Rotary(kv.ROTARY_HALVES if c["style"] == "halves" else kv.ROTARY_PAIRS, c["first"], c["dims"], s["table"])
    kv.nvfp4_kv_append(kv.Layout(c["h"], c["d"], c["t"]), s["k"], s["v"], s["slots"], s["kd"], s["ks"], s["vd"], s["vs"], q=s["q"],
                       q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"], rotary=rotary, positions=s["positions"],
                       k_global_scale=s["gk"], v_global_scale=s["gv"])
    return _append_outputs(s)


def _append_outputs(s):
    # the cache as its bytes, which have to be equal, and the rows of this call as the values that the cache holds for them
    return {x: s[x] for x in ("q_out", "k_out", "v_out", "kd", "ks", "vd", "vs")}


def _own_bounds(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_kv_page_bounds(kv.Layout(c["h"], c["d"], c["t"]), s["kd"], s["ks"], s["bounds"], s["bound_scales"], page_ids=s["pages"],
                            page_tokens=s["tokens"])
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _own_select(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_kv_select_pages(kv.Layout(c["h"], c["d"], c["t"]), s["q"], s["bounds"], s["bound_scales"], s["page_table"], s["lens"],
                             s["sel_table"], s["sel_lens"], sink_pages=c["sink"], recent_pages=c["recent"], sel_index=s["sel_index"],
                             scores=s["scores"])
    return {"table": s["sel_table"], "index": s["sel_index"], "lens": s["sel_lens"], "scores": s["scores"]}


def _own_attend(s):
    import nvfp4_paged_kv_gb300 as kv
    c = s["case"]
    kv.nvfp4_paged_sparse_decode_attention(kv.Layout(c["h"], c["d"], c["t"]), s["q"], s["kd"], s["ks"], s["gk"], s["vd"], s["vs"], s["gv"],
                                           s["sel_table"], s["sel_lens"], s["sm_scale"], s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _rotate(x, s):
    """x [rows, heads, d] in 32 bits, each product and each sum rounded once."""
    c = s["case"]
    if c["style"] == "none":
        return x
    first, r = c["first"], c["dims"]
    cos, sin = s["table"][s["positions"].long()][:, None].chunk(2, -1)
    part = x[..., first:first + r]
    a, b = part.chunk(2, -1) if c["style"] == "halves" else (part[..., 0::2], part[..., 1::2])
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.cat([a, b], -1) if c["style"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([x[..., :first], part, x[..., first + r:]], -1)


def _encode(x, g, e2m1):
    """Codes [.., d], scale bytes [.., d / 16] and the values that they stand for, of x in 32 bits."""
    blocks = x.unflatten(-1, (-1, 16))
    scale = (blocks.abs().amax(-1) / (g * 6)).clamp(max=448).to(torch.float8_e4m3fn)
    sg = scale.float() * g
    y = blocks * torch.where(sg == 0, 0.0, 1.0 / sg)[..., None]
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(torch.uint8)
    code = code | (torch.signbit(y).byte() << 3)
    value = e2m1[code.int()] * scale.float()[..., None] * g
    return code.flatten(-2), scale.view(torch.uint8), value.flatten(-2)


def _plain_append(s):
    t, rows = s["case"]["t"], s["real"]
    page, at = s["slots"] // t, s["slots"] % t
    s["q_out"][rows] = _rotate(s["q"].float(), s)[rows].to(torch.bfloat16)
    code, scale, value = _encode(_rotate(s["k"].float(), s), s["gk"], s["e2m1"])
    s["k_out"][rows] = value[rows].to(torch.bfloat16)
    s["kd"][page[rows], :, at[rows]] = (code[..., 0::2] | (code[..., 1::2] << 4))[rows]
    s["ks"][page[rows], :, at[rows]] = scale[rows]
    code, scale, value = _encode(s["v"].float(), s["gv"], s["e2m1"])
    s["v_out"][rows] = value[rows].to(torch.bfloat16)
    s["vs"][page[rows], :, at[rows] // 2, :, at[rows] % 2] = scale[rows]
    e, o = s["even"], s["odd"]
    s["vd"][page[e], :, at[e] // 2] = (s["vd"][page[e], :, at[e] // 2] & 0xF0) | code[e]
    s["vd"][page[o], :, at[o] // 2] = (s["vd"][page[o], :, at[o] // 2] & 0x0F) | (code[o] << 4)
    return _append_outputs(s)


def _keys(data, scales, e2m1):
    """K values without the tensor's scale: codes [.., t, d / 2] and scale bytes [.., t, d / 16] to [.., t, d]."""
    x = e2m1[torch.stack([data & 15, data >> 4], -1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _values(data, scales, e2m1):
    """V values: codes [.., t / 2, d] and scale bytes [.., t / 2, d / 16, 2] to [.., t, d]."""
    x = e2m1[torch.stack([data & 15, data >> 4], -2).int()]
    sc = scales.view(torch.float8_e4m3fn).float().movedim(-1, -2)
    return (x.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2).flatten(-3, -2)


def _plain_bounds(s):
    t, pages = s["case"]["t"], s["pages"].long()
    k = _keys(s["kd"][pages], s["ks"][pages], s["e2m1"])
    here = (torch.arange(t, device=k.device) < s["tokens"][:, None])[:, None, :, None]
    some = (s["tokens"] > 0)[:, None, None]
    top = torch.where(some, torch.where(here, k, -math.inf).amax(2), 0.0)
    low = torch.where(some, torch.where(here, k, math.inf).amin(2), 0.0)
    # (a number as the divisor would be turned into a product with its reciprocal)
    scale = torch.maximum(top.abs(), low.abs()).amax(-1, keepdim=True) / torch.full_like(k[:1, :1, 0, :1], 127)
    top = torch.where(scale > 0, (top / scale).ceil().clamp(max=127), 0.0)
    low = torch.where(scale > 0, (low / scale).floor().clamp(min=-127), 0.0)
    s["bounds"][pages] = torch.stack([top, low], 2).to(torch.int8)
    s["bound_scales"][pages] = scale[..., 0]
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _plain_select(s):
    c = s["case"]
    b, h, d, t, budget = c["b"], c["h"], c["d"], c["t"], c["budget"]
    maxp, dev = s["page_table"].shape[1], s["q"].device
    q = s["q"].float().view(b, h, -1, d)
    step = q.abs().amax(-1, keepdim=True) / torch.full_like(q[:1, :1, :1, :1], 255)
    qi = torch.where(step > 0, (q / step).round(), 0.0)
    ids, heads = s["page_table"].long()[:, None], torch.arange(h, device=dev)[:, None]
    hi, lo = s["bounds"][ids, heads].float().unbind(-2)
    total = torch.einsum("bhgd,bhpd->bhgp", qi.clamp(min=0), hi) + torch.einsum("bhgd,bhpd->bhgp", qi.clamp(max=0), lo)
    score = (total * step * s["bound_scales"][ids, heads][:, :, None]).amax(2)
    n = _pages(s["lens"], t)[:, None, None]
    at = torch.arange(maxp, device=dev)
    score = torch.where((at < c["sink"]) | (at >= n - c["recent"]), math.inf, score)
    s["scores"].copy_(torch.where(at < n, score, s["scores"]))
    order = torch.sort(torch.where(at < n, score, -math.inf), dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=maxp)
    count = n.clamp(max=budget)
    order = torch.where(torch.arange(budget, device=dev) < count, order, maxp).sort(-1).values
    kept = order < maxp
    s["sel_index"].copy_(torch.where(kept, order, -1))
    table = s["page_table"][:, None].expand(b, h, maxp).gather(2, order.clamp(max=maxp - 1))
    s["sel_table"].copy_(torch.where(kept, table, -1))
    last = s["lens"][:, None] - (n[..., 0] - 1) * t
    s["sel_lens"].copy_(torch.where(n[..., 0] > 0, (count[..., 0] - 1) * t + last, 0).expand(b, h))
    return {"table": s["sel_table"], "index": s["sel_index"], "lens": s["sel_lens"], "scores": s["scores"]}


def _plain_attend(s):
    c = s["case"]
    b, h, d = c["b"], c["h"], c["d"]
    ids, heads = s["sel_table"].long().clamp(min=0), torch.arange(h, device=s["q"].device)[:, None]
    k = _keys(s["kd"][ids, heads], s["ks"][ids, heads], s["e2m1"]).flatten(2, 3)
    q = s["q"].float().view(b, h, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (s["sm_scale"] * s["gk"])
    del k
    here = (torch.arange(x.shape[-1], device=x.device) < s["sel_lens"][..., None])[:, :, None]
    x = torch.where(here, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(here, torch.exp(x - top), 0.0)
    total = p.sum(-1, keepdim=True)
    v = _values(s["vd"][ids, heads], s["vs"][ids, heads], s["e2m1"]).flatten(2, 3)
    some = total > 0
    out = torch.where(some, torch.matmul(p, v) * s["gv"] / total, 0.0)
    s["out"].copy_(out.view(b, -1, d))
    s["lse"].copy_(torch.where(some, top + torch.log(total), -math.inf).view(b, -1))
    return {"out": s["out"], "lse": s["lse"]}


_OWN = {"append": _own_append, "bounds": _own_bounds, "select": _own_select, "attend": _own_attend}
_PLAIN = {"append": _plain_append, "bounds": _plain_bounds, "select": _plain_select, "attend": _plain_attend}


# ------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    return _WORK[case["op"]](case)


def _work_append(c):
    real, hq, h, d = c["rows"] - c["padding"], c["hq"], c["h"], c["d"]
    turned = 0 if c["style"] == "none" else c["dims"]
    spots = min(real, 32768)
    return {"bytes": real * ((hq + 2 * h) * d * 2 + (hq + 2 * h) * d * 2 + 2 * h * d * 9 / 16 + 12) + spots * turned * 4,
            "flops": real * ((hq + h) * turned * 3 + 2 * h * d * 4)}


def _work_bounds(c):
    real = 0.5 if c["partial"] else 1.0
    return {"bytes": c["pages"] * c["h"] * (c["t"] * real * c["d"] * 9 / 16 + 2 * c["d"] + 4), "flops": c["pages"] * c["h"] * c["t"] * real * c["d"] * 3}


def _mean_pages(c):
    return max(1.0, (c["low"] + c["high"]) / 2 / c["t"])


def _work_select(c):
    scored = c["b"] * c["h"] * _mean_pages(c)
    if _mean_pages(c) <= c["budget"]:  # every page is taken
        scored = c["b"] * c["h"]
    return {"bytes": scored * (2 * c["d"] + 8) + c["b"] * (c["hq"] * c["d"] * 2 + c["h"] * c["budget"] * 8),
            "flops": scored * c["hq"] / c["h"] * c["d"] * 2}


def _work_attend(c):
    tokens = c["b"] * c["h"] * c["t"] * min(c["budget"], _mean_pages(c))
    return {"bytes": tokens * c["d"] * 9 / 8 + c["b"] * c["hq"] * (c["d"] * 4 + 4), "flops": tokens * (c["hq"] // c["h"]) * c["d"] * 4}


_WORK = {"append": _work_append, "bounds": _work_bounds, "select": _work_select, "attend": _work_attend}


# ------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _f32(x):
    return x.float().double()


def _nearest(y, grid, even):
    """The entry of `grid` (ascending, from 0) nearest to y >= 0, a tie to the entry with an even number; over the last: the last."""
    at = torch.searchsorted(grid, y.clamp(max=grid[-1].item())).clamp(max=len(grid) - 1)
    below = (at - 1).clamp(min=0)
    up, down = grid[at] - y, y - grid[below]
    return torch.where((down < up) | ((down == up) & (even[below])), grid[below], grid[at])


def _stored(x, g):
    """The values that the cache holds for x [.., d]: the encoding's definition, its 32-bit roundings made in 64 bits."""
    dev = x.device
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=dev)
    e4m3 = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=dev)
    parts = []
    for block in x.unflatten(-1, (-1, 16)).split(512):
        want = _f32(block.abs().amax(-1) / _f32(6 * g))
        scale = _nearest(want, e4m3, torch.arange(127, device=dev) % 2 == 0)
        sg = _f32(scale * g)
        r = torch.where(sg > 0, _f32(1 / torch.where(sg > 0, sg, 1.0)), 0.0)[..., None]
        y = _f32(block * r)
        parts.append((torch.sign(y) * _nearest(y.abs(), e2m1, torch.arange(8, device=dev) % 2 == 0) * scale[..., None] * g).flatten(-2))
    return torch.cat(parts)


def _exact_append(s):
    c = s["case"]
    real = (s["slots"] >= 0)[:, None, None]

    def turned(x, each):
        x = x.double().clone()
        if c["style"] == "none":
            return x
        half = c["dims"] // 2
        i = torch.arange(half, device=x.device)
        one, two = (c["first"] + i, c["first"] + half + i) if c["style"] == "halves" else (c["first"] + 2 * i, c["first"] + 2 * i + 1)
        row = s["table"].double()[s["positions"].long()]
        cos, sin = row[:, None, :half], row[:, None, half:]
        a, b = x[..., one], x[..., two]
        x[..., one] = each(each(a * cos) - each(b * sin))
        x[..., two] = each(each(b * cos) + each(a * sin))
        return x

    q = turned(s["q"], lambda v: v)
    k = _stored(turned(s["k"], _f32), s["gk"].double())
    v = _stored(s["v"].double(), s["gv"].double())
    return {"q_out": torch.where(real, q, 0.0), "k_out": torch.where(real, k, 0.0), "v_out": torch.where(real, v, 0.0),
            "kd": None, "ks": None, "vd": None, "vs": None}


def _exact_bounds(s):
    """The scales: the largest magnitude among the page's tokens over 127."""
    pages, scales = s["pages"].long(), s["bound_scales"].double().clone()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=scales.device)
    for i in torch.arange(len(pages), device=scales.device).split(256):
        data = s["kd"][pages[i]]
        block = torch.maximum(mag[(data & 7).long()], mag[((data >> 4) & 7).long()]).unflatten(-1, (-1, 8)).amax(-1)
        top = (block * s["ks"][pages[i]].view(torch.float8_e4m3fn).double()).amax(-1)
        here = torch.arange(top.shape[-1], device=top.device) < s["tokens"][i][:, None, None]
        scales[pages[i]] = torch.where(here, top, 0.0).amax(-1) / 127
    return {"bounds": None, "scales": scales}


def _exact_select(s):
    c, scores = s["case"], s["scores"].double().clone()
    for b in range(c["b"]):
        n = -(-int(s["lens"][b]) // c["t"])
        lo, hi = min(c["sink"], n), max(0, n - c["recent"])
        scores[b, :, :n] = math.inf
        if hi <= lo:
            continue
        ids = s["page_table"][b, lo:hi].long()
        q = s["q"][b].double().view(c["h"], -1, c["d"])
        step = _f32(q.abs().amax(-1, keepdim=True) / torch.full_like(q[:1, :1, :1], 255))
        qi = torch.round(_f32(q / step.clamp(min=1e-300)))
        box = s["bounds"][ids].double().permute(1, 2, 0, 3)  # [h, 2, pages, d]
        pick = torch.matmul(qi.clamp(min=0), box[:, 0].transpose(1, 2)) + torch.matmul(qi.clamp(max=0), box[:, 1].transpose(1, 2))
        scores[b, :, lo:hi] = (pick * step * s["bound_scales"][ids].double().t()[:, None]).amax(1)
    return {"table": None, "index": None, "lens": None, "scores": scores}


def _exact_attend(s):
    c = s["case"]
    b, hq, h, d, t = c["b"], c["hq"], c["h"], c["d"], c["t"]
    grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=s["q"].device)
    out, lse = torch.zeros((b, hq, d), dtype=torch.float64, device=s["q"].device), torch.full((b, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    scale = float(torch.tensor(s["sm_scale"], dtype=torch.float32)) * s["gk"].double()
    lens = s["sel_lens"].cpu()
    for i in range(b):
        for j in range(h):
            n = int(lens[i, j])
            if n == 0:
                continue
            ids = s["sel_table"][i, j, :-(-n // t)].long()
            kd, vd = s["kd"][ids, j], s["vd"][ids, j]
            ks, vs = s["ks"][ids, j].view(torch.float8_e4m3fn).double(), s["vs"][ids, j].view(torch.float8_e4m3fn).double()
            k = torch.empty((len(ids), t, d), dtype=torch.float64, device=kd.device)
            k[..., 0::2], k[..., 1::2] = grid[(kd & 15).long()], grid[(kd >> 4).long()]
            k = (k * ks.repeat_interleave(16, -1)).reshape(-1, d)[:n]
            v = torch.empty((len(ids), t, d), dtype=torch.float64, device=kd.device)
            v[:, 0::2] = grid[(vd & 15).long()] * vs[..., 0].repeat_interleave(16, -1)
            v[:, 1::2] = grid[(vd >> 4).long()] * vs[..., 1].repeat_interleave(16, -1)
            g = slice(j * (hq // h), (j + 1) * (hq // h))
            x = s["q"][i, g].double() @ k.t() * scale
            lse[i, g] = torch.logsumexp(x, -1)
            out[i, g] = torch.exp(x - lse[i, g, None]) @ v.reshape(-1, d)[:n] * s["gv"].double()
    return {"out": out, "lse": lse}


_EXACT = {"append": _exact_append, "bounds": _exact_bounds, "select": _exact_select, "attend": _exact_attend}
