"""The decode-step operators on the host: what their argument checks refuse (nothing is launched; the
pointers are never dereferenced), sizes, and their plain forms against closed cases."""
import ctypes

import numpy as np
import pytest

import plain_steps


@pytest.fixture(scope="module")
def kv():
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


FAKE, MIS = 1 << 20, (1 << 20) + 8


def rotary(kv, **kw):
    r = kv.Rotary.__new__(kv.Rotary)
    ctypes.Structure.__init__(r, 0, 0, 64, 100, FAKE)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def append_args(kv, **kw):
    a = dict(layout=kv.Layout(8, 128, 64), src=kv.BF16, rows=4, hq=32, q=FAKE, qs=6144, k=FAKE + 64, ks=6144,
             v=FAKE + 128, vs=6144, slots=FAKE, rotary=rotary(kv), positions=FAKE, gk=None, gv=None,
             kd=FAKE, kss=FAKE, vd=FAKE, vss=FAKE, pages=8, out=kv.BF16, q_out=FAKE + 256, qos=4096,
             k_out=None, v_out=None, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), 1), (dict(hq=-1), 1), (dict(src=7), 1), (dict(out=5), 1), (dict(src=2), 2),
    (dict(out=2), 2), (dict(q=None), 1), (dict(q=MIS), 1), (dict(q_out=None), 1), (dict(q_out=FAKE), 1),
    (dict(qs=4088), 1), (dict(qs=4097), 1), (dict(ks=1016), 1), (dict(vs=1020), 1), (dict(k=None), 1),
    (dict(v=MIS), 1), (dict(slots=None), 1), (dict(positions=None), 1), (dict(pages=0), 1),
    (dict(kd=None), 1), (dict(kss=MIS), 1), (dict(vd=MIS), 1), (dict(vss=None), 1), (dict(k_out=MIS), 1),
    (dict(k_out=FAKE + 64), 1), (dict(v_out=FAKE + 128), 1), (dict(qos=4000), 1),
])
def test_append_refuses(kv, bad, code):
    assert kv.load().nvfp4_kv_append(*append_args(kv, **bad)) == code


@pytest.mark.parametrize("bad", [dict(style=2), dict(dims=0), dict(dims=48), dict(dims=160), dict(first_dim=-16),
                                 dict(first_dim=8), dict(first_dim=80), dict(max_positions=0),
                                 dict(cos_sin=None), dict(cos_sin=MIS)])
def test_append_refuses_rotations(kv, bad):
    assert kv.load().nvfp4_kv_append(*append_args(kv, rotary=rotary(kv, **bad))) == 1


@pytest.mark.parametrize("lay,code", [((8, 120, 64), 1), ((8, 96, 64), 2), ((8, 128, 33), 1), ((0, 128, 64), 1)])
def test_append_refuses_layouts(kv, lay, code):
    assert kv.load().nvfp4_kv_append(*append_args(kv, layout=kv.Layout(*lay))) == code


def test_no_rows_is_a_no_op(kv):
    assert kv.load().nvfp4_kv_append(*append_args(kv, rows=0, q=None, k=None, v=None, slots=None)) == 0
    lay = kv.Layout(8, 128, 64)
    assert kv.load().nvfp4_kv_page_bounds(lay, None, None, 0, None, None, 0, None, None, None, None) == 0
    assert kv.load().nvfp4_kv_select_pages(lay, 0, 32, None, None, None, 4, None, 4, None, 4, 1, 1, None, None,
                                           None, None, None, None) == 0
    assert kv.load().nvfp4_paged_sparse_decode_attention(lay, 0, 32, None, None, None, None, None, None, None, 4,
                                                         None, 4, None, 0.1, None, 0, None, None, None, None) == 0


def test_bounds_refuses(kv):
    f = kv.load().nvfp4_kv_page_bounds
    good = [kv.Layout(8, 128, 64), FAKE, FAKE, 8, None, None, 8, FAKE, FAKE, None, None]
    for at, bad, code in ((0, kv.Layout(8, 96, 64), 2), (0, kv.Layout(8, 120, 64), 1), (0, kv.Layout(8, 128, 40), 2), (1, None, 1), (1, MIS, 1),
                          (2, MIS, 1), (3, 0, 1), (6, -1, 1), (6, 9, 1), (7, None, 1), (7, MIS, 1), (8, None, 1)):
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)


def test_select_refuses(kv):
    f = kv.load().nvfp4_kv_select_pages
    good = [kv.Layout(8, 128, 64), 2, 32, FAKE, FAKE, FAKE, 8, FAKE, 100, FAKE, 10, 1, 1, FAKE, FAKE, None, None,
            None, None]
    for at, bad, code in ((0, kv.Layout(8, 96, 64), 2), (1, -1, 1), (2, 0, 1), (2, 30, 2), (2, 72, 2), (3, MIS, 1),
                          (3, None, 1), (4, MIS, 1), (5, None, 1), (6, 0, 1), (7, None, 1), (8, 0, 1),
                          (8, 49152 + 1, 2), (9, None, 1), (10, 0, 1), (10, 1, 1), (11, -1, 1), (11, 10, 1),
                          (12, 0, 1), (12, 11, 1), (13, None, 1), (14, None, 1), (1, 8192, 2),
                          (10, 1 << 30, 2), (0, kv.Layout(8, 128, 1 << 28), 2)):
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)


def test_sparse_decode_refuses(kv):
    f = kv.load().nvfp4_paged_sparse_decode_attention
    lay = kv.Layout(8, 128, 64)
    need = kv.nvfp4_paged_sparse_decode_workspace_size(lay, 2, 32, 10)
    good = [lay, 2, 32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, FAKE, 10, FAKE, 0.1, FAKE, need, FAKE, None,
            None, None]
    for at, bad, code in ((0, kv.Layout(8, 96, 64), 2), (0, kv.Layout(8, 128, 40), 2), (1, -1, 1), (1, 8192, 2),
                          (2, 0, 1), (2, 30, 2), (2, 72, 2), (3, MIS, 1), (4, None, 1), (5, MIS, 1), (6, None, 1),
                          (7, MIS, 1), (9, None, 1), (10, 0, 1), (11, None, 1), (12, 0, 1), (13, None, 1),
                          (15, None, 3), (15, MIS, 3), (16, need - 1, 3), (17, None, 1), (17, MIS, 1),
                          (12, 1 << 25, 2)):
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)
    assert kv.nvfp4_paged_sparse_decode_workspace_size(lay, 8192, 32, 10) == 0
    assert kv.nvfp4_paged_sparse_decode_workspace_size(lay, 2, 30, 10) == 0
    assert kv.nvfp4_paged_sparse_decode_workspace_size(lay, 2, 32, 0) == 0


def test_binding_refuses_tensors_on_the_host(kv):
    import torch
    k = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    b = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)  # noqa: E731
    lay = kv.Layout(8, 128, 64)
    pool = [b(1, 8, 64, 64), b(1, 8, 64, 8), b(1, 8, 64, 64), b(1, 8, 64, 8)]
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_kv_append(lay, k, k, torch.zeros(2, dtype=torch.int64), *pool)
    with pytest.raises(TypeError, match="dtype"):
        kv.nvfp4_kv_append(lay, k, k.half(), torch.zeros(2, dtype=torch.int64), *pool)
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_kv_page_bounds(lay, pool[0], pool[1], i8(1, 8, 2, 128), torch.zeros(1, 8))
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_kv_select_pages(lay, k, i8(1, 8, 2, 128), torch.zeros(1, 8), i(2, 5), i(2), i(2, 8, 2), i(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        kv.nvfp4_paged_sparse_decode_attention(lay, k, pool[0], pool[1], None, pool[2], pool[3], None, i(2, 8, 2),
                                               i(2, 8), 0.1, k)
    with pytest.raises(ValueError):
        kv.Rotary(kv.ROTARY_HALVES, 0, 64, torch.zeros(4, 32))


# ------------------------------------------------------------------ the plain forms on closed cases

def test_plain_rotation_by_a_quarter_turn():
    x = np.arange(1, 33, dtype=np.float64)[None]
    row = np.concatenate([np.zeros(16), np.ones(16)])   # cos 0, sin 1: (a, b) -> (-b, a)
    y = plain_steps.rotate(x, row, "halves", 0, 32)
    assert np.array_equal(y[0, :16], -x[0, 16:]) and np.array_equal(y[0, 16:], x[0, :16])
    y = plain_steps.rotate(x, row, "pairs", 0, 32)
    assert np.array_equal(y[0, 0::2], -x[0, 1::2]) and np.array_equal(y[0, 1::2], x[0, 0::2])


def test_plain_encode_equals_the_oracle():
    import oracle
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((4, 2, 4, 64)) * 10.0 ** rng.integers(-3, 3, (4, 2, 4, 1))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)                  # truncated to BF16
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    g = np.float32(np.abs(x).max() / 2688)
    data, scales = oracle.quantize_pages(bits, oracle.BF16, 2, 64, 4, g)
    code, sb = plain_steps.encode(x.astype(np.float64), g)
    assert np.array_equal(code[..., 0::2] | (code[..., 1::2] << 4), data.reshape(4, 2, 4, 32))
    assert np.array_equal(sb, scales.reshape(4, 2, 4, 4))


def test_plain_attention_equals_the_oracle():
    """One table for all heads: the per-head form is the dense one."""
    import oracle
    rng = np.random.default_rng(1)
    P, H, T, D, G, B = 6, 2, 16, 64, 3, 2
    kd, vd = (rng.integers(0, 256, (P, H, T, D // 2)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.integers(0x28, 0x39, (P, H, T, D // 16)).astype(np.uint8) for _ in range(2))
    qb = (rng.standard_normal((B, H * G, D)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    q = (qb.astype(np.uint32) << 16).view(np.float32)
    table, lens = np.array([[3, 1, 5], [0, 2, 4]], np.int32), np.array([40, 17], np.int32)
    want, want_lse = oracle.paged_decode_attention(qb, kd, ks, 1.0, vd, vs, 0.5, table, lens, 0.125, H, T,
                                                   v_packing=oracle.TOKEN_PAIRS)
    per = np.repeat(table[:, None], H, 1)
    got, lse = plain_steps.attend(q, kd, ks, vd.reshape(P, H, T // 2, D), vs.reshape(P, H, T // 2, D // 16, 2), 1.0,
                                  0.5, per, np.repeat(lens[:, None], H, 1), T, 0.125)
    assert np.abs(got - want).max() < 1e-6 and np.abs(lse - want_lse).max() < 1e-6


def test_plain_bounds_hold_every_key():
    rng = np.random.default_rng(2)
    kd = rng.integers(0, 256, (3, 32, 32)).astype(np.uint8)
    ks = rng.integers(0, 0x7F, (3, 32, 4)).astype(np.uint8)
    hi, lo, s = plain_steps.page_bounds(kd, ks, 30)
    v = plain_steps.keys(kd, ks)[:, :30]
    unit = s[:, None, None] * (1 + 2.0 ** -22)
    assert (v <= np.where(hi < 0, hi / (1 + 2.0 ** -22) ** 2, hi)[:, None] * unit).all()
    assert (v >= np.where(lo > 0, lo / (1 + 2.0 ** -22) ** 2, lo)[:, None] * unit).all()
