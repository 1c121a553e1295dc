"""The bound that the window decodes are held to, on the CPU: it takes the exact values rounded to BF16, and refuses wrong ones
(with the right log-sum-exp beside them)."""
import numpy as np
import pytest
import torch

import window_values


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D,case", [(64, 0), (64, 1), (64, 2), (128, 1), (256, 2)])
def test_wrong_values_are_refused(fmt, D, case):
    lens, window, sinks = window_values.LONG[case]
    c = window_values.Leaning("cpu", fmt, lens, 1, 64, D, 4, window, sinks, seed=len(lens))
    out, lse = window_values.exact(c)
    bf16 = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731
    window_values.check(c, (bf16(out), lse))
    for wrong in (0 * out, -out, 2 * out, out[:, ::-1].copy(), np.roll(out, 1, -1), out * 0.9, window_values.exact(c, 8)[0], window_values.exact(c, 30)[0]):
        with pytest.raises(AssertionError):
            window_values.check(c, (bf16(wrong), lse))
