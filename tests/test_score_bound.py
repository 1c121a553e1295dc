"""What the page score promises (its plain form; the GPU's scores equal it bit for bit): it is at least the product of
the rounded query with every key of the page, and the query's own product lies above it by no more than half a step
of the query in every dim."""
import numpy as np
import pytest

import plain_steps


def page(rng, T, D, lo=0x18, hi=0x45):
    return rng.integers(0, 256, (1, T, D // 2)).astype(np.uint8), rng.integers(lo, hi, (1, T, D // 16)).astype(np.uint8)


def score_of(q, kd, ks):
    """Score, and its slack, of one page (tokens all valid) for one query [D]; the keys [T, D]."""
    hi, lo, s = plain_steps.page_bounds(kd, ks, kd.shape[1])
    bounds = np.stack([np.zeros_like(hi), hi])[:, :, None], np.stack([np.zeros_like(lo), lo])[:, :, None]
    # three pages in the table: the last is always taken, so the one of interest is scored
    box = np.concatenate(bounds, 2)[[1, 0, 0]]
    scales = np.stack([s, s, s]).astype(np.float64)
    _, _, _, scores = plain_steps.select(q[None, None], box, scales, np.arange(3)[None], np.array([48]), 16, 2, 0, 1)
    f = plain_steps.f32(np.abs(q).max() / 255)
    far = np.maximum(np.abs(hi[0].astype(np.float64)), np.abs(lo[0])) * float(s[0])
    return scores[0, 0, 0], f, far, plain_steps.keys(kd, ks)[0]


def bf16(x):
    return (np.asarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("outlier", [1.0, 20.0, 300.0, 1e6])
def test_score_bounds_the_products_up_to_the_querys_rounding(D, outlier):
    rng = np.random.default_rng(D + int(outlier))
    above = 0
    for _ in range(60):
        kd, ks = page(rng, int(rng.choice([1, 2, 16])), D)
        q = bf16(rng.standard_normal(D))
        q[rng.integers(D)] *= outlier
        q = bf16(q)
        score, f, far, keys = score_of(q, kd, ks)
        # |q - f q_i| <= f/2, and 2^-16 f for the FP32 quotient q / f <= 255; bounds and score are FP32 products
        product, rounding = (keys @ q).max(), 2.0 ** -21 * (np.abs(q) + f) @ far
        assert product <= score + (0.5 + 2.0 ** -16) * f * far.sum() + rounding
        qi = np.rint(plain_steps.f32(q / f))
        assert (keys @ (f * qi)).max() <= score + rounding
        above += product > score
    if outlier == 300.0:
        assert above > 0   # the slack is needed


def test_small_query_dims_beside_a_large_one_count_as_zero():
    """One dim of 255 and 63 of 0.4375, keys of all sixes: a score of 1530 for a product of 1695."""
    kd, ks = np.full((1, 16, 32), 0x77, np.uint8), np.full((1, 16, 4), 0x38, np.uint8)
    q = np.full(64, 0.4375)
    q[0] = 255.0
    score, f, far, keys = score_of(q, kd, ks)
    assert f == 1.0 and abs(score - 1530) < 1e-3
    assert (keys @ q).max() == 255 * 6 + 63 * 0.4375 * 6 == 1695.375
    assert 1695.375 <= score + 0.5 * f * far.sum()
