"""Values of the decodes over long windows, cut into pieces and joined, within a bound that wrong values do not pass
(test_window_values)."""
import pytest
import torch

import window_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(window_values.LONG)))
def test_long_windows(kv, cuda, fmt, D, case):
    lens, window, sinks = window_values.LONG[case]
    c = window_values.Leaning(cuda, fmt, lens, 1, 64, D, 4, window, sinks, seed=len(lens))
    size = (kv.nvfp4_paged_fp8_decode_workspace_size if fmt == "fp8" else kv.nvfp4_paged_window_decode_workspace_size)
    ws = torch.randint(0, 256, (size(c.layout(kv), len(lens), 4, c.maxp),), dtype=torch.uint8, device=cuda)
    window_values.check(c, c.run(kv, workspace=ws))


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D,H,G,T", [(64, 2, 8, 16), (128, 8, 4, 64), (256, 2, 3, 48)])
def test_a_batch(kv, cuda, fmt, D, H, G, T):
    for window, sinks in ((700, 5), (64, 0), (5000, 0)):
        c = window_values.Leaning(cuda, fmt, [5000, 1, 0, 333, 2048, 701, 64, 4095], H, T, D, G, window, sinks, seed=T)
        window_values.check(c, c.run(kv))
