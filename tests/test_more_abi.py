"""The step tables, the FP8 pages and the attentions over them and with a sliding window on the host: what their argument
checks refuse (nothing is launched; the pointers are never dereferenced), sizes, and their plain forms on closed cases."""
import numpy as np
import pytest

import plain_windows


@pytest.fixture(scope="module")
def kv():
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


FAKE, MIS = 1 << 20, (1 << 20) + 8


def refuses(f, good, cases):
    for at, bad, code in cases:
        a = list(good.values())
        a[list(good).index(at)] = bad
        assert f(*a) == code, (at, bad, code)


def test_step_tables_refuses(kv):
    good = dict(layout=kv.Layout(1, 64, 16), batch=4, past=FAKE, new=FAKE, stack=FAKE, capacity=100, count=FAKE, left=FAKE,
                table=FAKE, maxp=8, lens=FAKE, starts=FAKE, slots=FAKE, positions=FAKE, rows=32, full=FAKE, full_cap=6,
                status=None, stream=None)
    refuses(kv.load().nvfp4_kv_step_tables, good, [
        ("layout", None, 1), ("layout", kv.Layout(1, 64, 0), 1), ("batch", -1, 1), ("batch", 8193, 1), ("past", None, 1),
        ("new", None, 1), ("stack", None, 1), ("capacity", -1, 1), ("count", None, 1), ("left", None, 1), ("table", None, 1),
        ("maxp", 0, 1), ("maxp", 1 << 27, 2), ("lens", None, 1), ("starts", None, 1), ("slots", None, 1), ("positions", None, 1),
        ("rows", -1, 1), ("full_cap", 5, 1), ("full_cap", -1, 1)])
    good["full_cap"] = 10000
    refuses(kv.load().nvfp4_kv_step_tables, good, [("batch", 8193, 2)])
    assert kv.load().nvfp4_kv_step_tables(*[0 if k == "batch" else v for k, v in good.items()]) == 0


def test_fp8_pages_refuses(kv):
    good = dict(layout=kv.Layout(8, 128, 64), kind=kv.BF16, src=FAKE, scales=None, g=None, pool=8, ids=FAKE, tokens=None, dst=2 * FAKE,
                dst_scales=FAKE, dst_pool=8, dst_ids=FAKE, num=4, status=None, stream=None)
    f = kv.load().nvfp4_kv_fp8_pages
    refuses(f, good, [
        ("layout", None, 1), ("layout", kv.Layout(8, 120, 64), 1), ("kind", 4, 1), ("kind", -1, 1), ("kind", kv.FP8_E4M3, 2),
        ("src", None, 1), ("src", MIS, 1), ("src", 2 * FAKE, 1), ("pool", 0, 1), ("dst", None, 1), ("dst", MIS, 1),
        ("dst_scales", None, 1), ("dst_pool", 0, 1), ("num", -1, 1), ("layout", kv.Layout(1, 1 << 17, 16), 2),
        ("layout", kv.Layout(1, 256, 1 << 22), 2)])
    refuses(f, dict(good, ids=None), [("num", 9, 1)])
    refuses(f, dict(good, dst_ids=None), [("num", 9, 1)])
    packed = dict(good, kind=kv.NVFP4, scales=FAKE)
    refuses(f, packed, [("scales", None, 1), ("scales", MIS, 1), ("layout", kv.Layout(8, 128, 64, 2), 1),
                        ("layout", kv.Layout(8, 128, 33, kv.PACK_TOKEN_PAIRS), 1)])
    assert f(*[0 if k == "num" else None if k in ("src", "dst", "dst_scales") else v for k, v in good.items()]) == 0


def decode_args(kv, fmt):
    lay = kv.Layout(8, 128, 64)
    need = (kv.nvfp4_paged_fp8_decode_workspace_size if fmt == "fp8" else kv.nvfp4_paged_window_decode_workspace_size)(lay, 2, 32, 10)
    return dict(layout=lay, batch=2, hq=32, q=FAKE, kd=FAKE, ks=FAKE, gk=FAKE, vd=FAKE, vs=FAKE, gv=FAKE, pool=8, table=FAKE, maxp=10,
                lens=FAKE, window=100, sinks=4, sm=0.1, ws=FAKE, need=need, out=FAKE, lse=None, status=None, stream=None)


DECODE = [("batch", -1, 1), ("batch", 65536, 2), ("hq", 0, 1), ("hq", 30, 2), ("hq", 72, 2), ("q", None, 1), ("q", MIS, 1), ("kd", None, 1),
          ("kd", MIS, 1), ("vd", None, 1), ("vd", MIS, 1), ("pool", 0, 1), ("table", None, 1), ("maxp", 0, 1), ("maxp", 1 << 26, 2),
          ("lens", None, 1), ("window", -1, 1), ("sinks", -1, 1), ("ws", None, 3), ("ws", MIS, 3), ("need", 100, 3), ("out", None, 1),
          ("out", MIS, 1)]


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_decodes_refuse(kv, fmt):
    good = decode_args(kv, fmt)
    f = kv.load().nvfp4_paged_fp8_decode_attention if fmt == "fp8" else kv.load().nvfp4_paged_window_decode_attention
    refuses(f, good, DECODE + [("layout", kv.Layout(8, 96, 64), 2), ("layout", kv.Layout(8, 128, 40), 2), ("layout", kv.Layout(8, 120, 64), 1),
                               ("need", good["need"] - 1, 3)])
    if fmt == "nvfp4":
        refuses(f, good, [("window", 0, 1), ("ks", None, 1), ("vs", MIS, 1), ("gk", None, 1), ("gv", None, 1)])
    assert f(*[0 if k == "batch" else v for k, v in good.items()]) == 0
    size = kv.nvfp4_paged_fp8_decode_workspace_size if fmt == "fp8" else kv.nvfp4_paged_window_decode_workspace_size
    for bad in ((kv.Layout(8, 96, 64), 2, 32, 4), (kv.Layout(8, 128, 64), 2, 30, 4), (kv.Layout(8, 128, 64), 2, 72, 4),
                (kv.Layout(8, 128, 64), -1, 32, 4), (kv.Layout(8, 128, 64), 2, 32, 0)):
        assert size(*bad) == 0


def test_extend_refuses(kv):
    lay = kv.Layout(8, 128, 64)
    need = kv.nvfp4_paged_extend_attention_workspace_size(lay, 2, 32)
    good = dict(layout=lay, batch=2, rows=9, hq=32, q=FAKE, qs=6144, starts=FAKE, k=FAKE, kb=None, ks=None, v=FAKE, vb=None, vs=None, pool=8,
                table=FAKE, maxp=10, lens=FAKE, window=0, sinks=0, sm=0.1, ws=FAKE, need=need, out=2 * FAKE, outs=4096, lse=None,
                status=None, stream=None)
    f = kv.load().nvfp4_paged_extend_attention
    refuses(f, good, [
        ("layout", None, 1), ("layout", kv.Layout(8, 96, 64), 2), ("layout", kv.Layout(8, 128, 40), 2), ("batch", -1, 1), ("batch", 65536, 2),
        ("rows", -1, 1), ("hq", 0, 1), ("hq", 30, 2), ("hq", 72, 2), ("q", None, 1), ("q", MIS, 1), ("qs", 4088, 1), ("qs", 4097, 1),
        ("starts", None, 1), ("k", None, 1), ("k", MIS, 1), ("v", None, 1), ("v", MIS, 1), ("pool", 0, 1), ("table", None, 1), ("maxp", 0, 1),
        ("maxp", 1 << 25, 2), ("lens", None, 1), ("window", -1, 1), ("sinks", -1, 1), ("ws", None, 3), ("ws", MIS, 3), ("need", need - 1, 3),
        ("out", None, 1), ("out", MIS, 1), ("out", FAKE, 1), ("outs", 4088, 1), ("outs", 4100, 1)])
    for none in ("batch", "rows"):
        assert f(*[0 if k == none else v for k, v in good.items()]) == 0
    assert kv.nvfp4_paged_extend_attention_workspace_size(kv.Layout(8, 96, 64), 2, 32) == 0
    assert kv.nvfp4_paged_extend_attention_workspace_size(lay, 2, 30) == 0


def test_binding_refuses_tensors_on_the_host(kv):
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    lay = kv.Layout(8, 128, 64)
    q = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    pool = b(1, 8, 64, 128)
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_kv_step_tables(lay, i(2), i(2), i(5), i(1), i(2, 4), i(2), i(3), torch.zeros(4, dtype=torch.int64), i(4))
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_kv_fp8_pages(lay, torch.zeros(1, 8, 64, 128, dtype=torch.bfloat16), pool, torch.zeros(1, 8))
    with pytest.raises(TypeError, match="dst"):
        kv.nvfp4_kv_fp8_pages(lay, torch.zeros(1, 8, 64, 128, dtype=torch.bfloat16), pool.short(), torch.zeros(1, 8))
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_paged_fp8_decode_attention(lay, q, pool, pool, i(2, 4), i(2), 0.1, q)
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_paged_window_decode_attention(lay, q, b(1, 8, 64, 64), b(1, 8, 64, 8), None, b(1, 8, 64, 64), b(1, 8, 64, 8), None, i(2, 4),
                                               i(2), 0.1, q, window=5)
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_paged_extend_attention(lay, q, pool, pool, i(2, 4), i(2), i(3), 0.1, q.clone())
    with pytest.raises(TypeError, match="bfloat16"):
        kv.nvfp4_paged_extend_attention(lay, q.half(), pool, pool, i(2, 4), i(2), i(3), 0.1, q)


# ------------------------------------------------------------------ the plain forms on closed cases

def test_plain_step_tables_by_hand():
    # T = 4: sequence 0 has 3 tokens on page 9 and adds 6; 1 ended with pages 5, 6; 2 adds 4 to nothing
    got = plain_windows.step_tables([3, 7, 0], [6, -1, 4], [2, 3, 0, 0], 2, [[9, -1, -1], [5, 6, -1], [-1, -1, -1]], 4, 12, 6)
    assert got["stack"] == [2, 3, 5, 6] and got["left"] == 1 and got["status"] == 0
    assert got["table"] == [[9, 6, 5], [5, 6, -1], [3, -1, -1]] and got["lens"] == [9, 0, 4] and got["starts"] == [0, 6, 6, 10]
    assert got["slots"] == [39, 24, 25, 26, 27, 20, 12, 13, 14, 15, -1, -1] and got["positions"] == [3, 4, 5, 6, 7, 8, 0, 1, 2, 3, 0, 0]
    assert got["full"] == [9, 6, 3, -1, -1, -1]


def test_plain_step_tables_agree_with_the_vectorised_form():
    """The measured plain form in torch operations against the loops."""
    import random

    import torch

    from perf import more_operators
    for seed in range(40):
        r = random.Random(seed)
        B, T, maxp = r.randint(1, 20), r.choice((1, 4, 16)), r.randint(1, 6)
        past = [r.randint(0, maxp * T) for _ in range(B)]
        new = [r.choice((-1, 0, min(1, maxp * T - p), r.randint(0, maxp * T - p))) for p in past]
        have = [-(-p // T) for p in past]
        ids = list(range(sum(have) + r.randint(0, 60)))
        r.shuffle(ids)
        table = [[ids.pop() for _ in range(n)] + [-1] * (maxp - n) for n in have]
        stack, rows = ids + [-1] * (sum(have) + 3), sum(max(a, 0) for a in new) + 4
        i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        s = {"case": {"t": T}, "past": i(past), "new": i(new), "table": i(table), "stack": i(stack), "count": i([len(ids)]), "left": i([0]),
             "lens": i([0] * B), "starts": i([0] * (B + 1)), "slots": torch.zeros(rows, dtype=torch.int64), "positions": i([0] * rows),
             "full": i([0] * (B + rows // T))}
        more_operators._plain_tables(s)
        want = plain_windows.step_tables(past, new, stack, len(ids), table, T, rows, B + rows // T)
        for name, x in want.items():
            if name != "status":
                got = s[name].tolist()
                assert (got if isinstance(x, list) else got[0]) == x, (seed, name)


def test_plain_fp8_page():
    x = np.zeros((2, 4, 16))
    x[0, 1, 3], x[0, 2, 0], x[0, 3, 5] = -2.0, 0.5, 100.0   # the last token does not count
    code, s = plain_windows.fp8_page(x, 3)
    assert s[1] == 1 and s[0] == np.float32(2 / 448) and (code[:, 3] == 0).all() and (code[1] == 0).all()
    assert plain_windows.FP8[code[0, 1, 3]] == -448 and plain_windows.FP8[code[0, 2, 0]] == 112


def test_plain_attention_of_one_visible_token():
    v = np.arange(12.0).reshape(4, 3)
    out, lse = plain_windows.attention(np.ones((2, 3)), np.ones((4, 3)), v, plain_windows.visible([0, 3], 4, 1, 0), 0.5)
    assert np.array_equal(out, v[[0, 3]]) and np.allclose(lse, 1.5)
    assert plain_windows.visible([5], 6, 2, 1).tolist() == [[True, False, False, False, True, True]]


@pytest.mark.parametrize("D", [64, 128])
def test_the_bound_tells_a_wrong_scale_of_one_tile(D):
    """The bound of the attention tests refuses an output computed with one V scale of 16 tokens in 1024 doubled."""
    g = np.random.default_rng(D)
    q, k, v = g.standard_normal((2, D)), g.standard_normal((1024, D)), g.standard_normal((1024, D))
    here = np.ones((2, 1024), bool)
    import torch

    def rounded(v):
        out, lse = plain_windows.attention(q, k, v, here, D ** -0.5)
        return torch.from_numpy(out).to(torch.bfloat16).double().numpy(), lse
    plain_windows.check(rounded(v), q, k, v, here, D ** -0.5, 4.0, blocks=True)
    w = v.copy()
    w[16:32] *= 2
    with pytest.raises(AssertionError):
        plain_windows.check(rounded(w), q, k, v, here, D ** -0.5, 4.0, blocks=True)
