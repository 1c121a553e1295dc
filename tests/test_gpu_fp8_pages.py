"""Pages encoded as FP8 with a scale for each page and head: every byte and scale equal to the definition's."""
import numpy as np
import pytest
import torch

import plain_steps
import plain_windows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def source(kind, P, H, T, D, g, dev):
    """Source pages: tensors for the call, and their values [P, H, T, D] in 64 bits."""
    if kind in ("bf16", "fp16"):
        x = torch.randn((P, H, T, D), generator=g) * 2.0 ** torch.randint(-12, 6, (P, H, 1, 1), generator=g)
        x = x.to({"bf16": torch.bfloat16, "fp16": torch.float16}[kind])
        return {"src": x.to(dev)}, x.double().numpy()
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
    scale = float(np.float32(0.037))
    if kind == "nvfp4":
        data, sc = u(0, 256, P, H, T, D // 2), u(0, 0x7F, P, H, T, D // 16)
        x = plain_steps.keys(data.numpy(), sc.numpy())
    else:
        data, sc = u(0, 256, P, H, T // 2, D), u(0, 0x7F, P, H, T // 2, D // 16, 2)
        x = values(data.numpy(), sc.numpy())
    return ({"src": data.to(dev), "src_scales": sc.to(dev), "global_scale": torch.tensor([scale], device=dev)},
            plain_steps.f32(x * scale))


def values(vd, vs):
    """V values of codes [.., T/2, D] and scale bytes [.., T/2, D/16, 2]."""
    code = np.stack([vd & 15, vd >> 4], -2)
    v = plain_steps.E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    sc = np.append(plain_steps.E4M3, 0.0)[np.moveaxis(vs, -1, -2) & 127]
    v = v.reshape(*v.shape[:-1], -1, 16) * sc[..., None]
    return v.reshape(*vd.shape[:-2], -1, vd.shape[-1])


def run(kv, dev, kind, P, H, T, D, ids, to, tokens, pool, seed=0, x=None, **kw):
    g = torch.Generator().manual_seed(seed)
    args, want = source(kind, P, H, T, D, g, dev) if x is None else x
    i = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    dst = torch.full((pool, H, T, D), 0x55, dtype=torch.uint8, device=dev)
    scales = torch.full((pool, H), -5.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    src = args.pop("src")
    lay = kv.Layout(H, D, T, kv.PACK_TOKEN_PAIRS if kind == "pairs" else kv.PACK_DIM_PAIRS)
    kv.nvfp4_kv_fp8_pages(lay, src, dst, scales, src_page_ids=i(ids), dst_page_ids=i(to), page_tokens=i(tokens), status=status, **args, **kw)
    torch.cuda.synchronize()
    n = len(ids if ids is not None else to if to is not None else range(P))
    code, s = np.full((pool, H, T, D), 0x55, np.uint8), np.full((pool, H), -5.0)
    for e in range(n):
        a, b = (e if ids is None else ids[e]), (e if to is None else to[e])
        m = T if tokens is None else tokens[e]
        if 0 <= a < P and 0 <= b < pool and 0 <= m <= T:
            code[b], s[b] = plain_windows.fp8_page(want[a], m)
    got = dst.cpu().numpy()
    assert np.array_equal(scales.double().cpu().numpy(), s)
    assert np.array_equal(got, code), np.argwhere(got != code)[:5]
    return int(status.item())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "nvfp4", "pairs"])
@pytest.mark.parametrize("H,T,D", [(2, 64, 128), (1, 16, 64), (3, 16, 256), (1, 128, 128), (2, 6, 16), (1, 2, 48), (1, 130, 256),
                                   (1, 512, 256), (5, 32, 80)])
def test_pages(kv, cuda, kind, H, T, D):
    """Partial, empty and full pages, gathered and scattered."""
    P = 6
    assert run(kv, cuda, kind, P, H, T, D, [5, 0, 2, 3], [1, 7, 0, 4], [T, 0, 1, T - 1], 8, seed=T + D) == 0


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
@pytest.mark.parametrize("T,D", [(1, 16), (3, 16), (1, 48), (5, 144)])
def test_runs_of_an_odd_number_of_blocks(kv, cuda, kind, T, D):
    assert run(kv, cuda, kind, 4, 3, T, D, None, [3, 2, 1, 0], [T, 0, (T + 1) // 2, T], 4) == 0


@pytest.mark.parametrize("kind", ["bf16", "pairs"])
def test_all_pages_without_lists(kv, cuda, kind):
    assert run(kv, cuda, kind, 9, 4, 32, 64, None, None, None, 9) == 0


def test_bad_entries_are_skipped_and_padding_is_silent(kv, cuda):
    assert run(kv, cuda, "bf16", 4, 2, 16, 64, [0, -1, 2, 1], [3, 2, -1, 1], None, 5) == 0
    assert run(kv, cuda, "bf16", 4, 2, 16, 64, [0, 4, 2, 1], [3, 2, 1, 0], None, 5) == kv.STATUS_PAGE_OOB
    assert run(kv, cuda, "nvfp4", 4, 2, 16, 64, [0, 3, 2, 1], [3, 5, 1, 0], None, 5) == kv.STATUS_PAGE_OOB
    assert run(kv, cuda, "pairs", 4, 2, 16, 64, [0, 3, 2, 1], [3, 2, 1, 0], [16, 17, -1, 2], 5) == kv.STATUS_BAD_SEQ_LEN


def test_zeros_tiny_and_huge_values(kv, cuda):
    """A page of zeros has scale 1; so has one whose largest value over 448 is below 2^-100; BF16's largest stays finite."""
    H, T, D = 1, 16, 64
    x = torch.zeros((6, H, T, D), dtype=torch.bfloat16)
    x[1] = 448 * 2.0 ** -101
    x[2] = 448 * 2.0 ** -100
    x[3] = torch.finfo(torch.bfloat16).max
    x[4, 0, 3, 5], x[4, 0, 3, 6] = -1.0, 1e-6
    x[5, 0, 0, 0] = -0.0
    assert run(kv, cuda, "bf16", 6, H, T, D, None, None, None, 6, x=({"src": x.to(cuda)}, x.double().numpy())) == 0


def test_hidden_tokens_may_be_anything(kv, cuda):
    """NaN and infinities past the valid tokens neither reach the scale nor the codes."""
    H, T, D = 2, 16, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn((2, H, T, D), generator=g).to(torch.bfloat16)
    y = x.clone()
    y[:, :, 9:] = float("nan")
    y[:, :, 12] = float("inf")
    assert run(kv, cuda, "bf16", 2, H, T, D, None, None, [9, 9], 2, x=({"src": y.to(cuda)}, x.double().numpy())) == 0
