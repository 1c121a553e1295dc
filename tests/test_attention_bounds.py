"""The bound that the GPU attention tests hold outputs to is narrow enough to see a mistake in one tile."""
import pytest
import torch

import plain_steps
from test_gpu_attention_numerics import Pool


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_bound_tells_a_wrong_scale_of_one_tile(D):
    """The same bound refuses an output computed with one V block scale of 16 tokens doubled in a pair of 2048 (on the
    host: the oracle's side carries the mistake)."""
    T, pages = 16, 128
    c = Pool("cpu", pages, 1, T, D, D)
    q = torch.randn((1, 2, D), generator=c.g).to(torch.bfloat16)
    table, lens = torch.arange(pages, dtype=torch.int32)[None, None], torch.tensor([[pages * T]], dtype=torch.int32)

    def exact():
        out, lse = plain_steps.attend(q.double().numpy(), c.kd.numpy(), c.ks.numpy(), c.vd.numpy(), c.vs.numpy(), c.gk, c.gv,
                                      table.numpy(), lens.numpy(), T, c.sm)
        return torch.from_numpy(out).to(torch.bfloat16).double().numpy(), lse
    good = exact()
    c.check(good, q, table, lens)
    c.vs[77] += 8   # one step of the exponent
    bad = exact()
    c.vs[77] -= 8
    with pytest.raises(AssertionError):
        c.check(bad, q, table, lens)
