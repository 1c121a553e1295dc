"""Optional scalars of the decode-step calls: an empty tensor is refused, not taken for an argument left out (its data
pointer is null, which means a scale of 1, or no status). On the host, through stand-ins for the library and tensors."""
import pytest
import torch

import nvfp4_paged_kv_gb300 as kv
from test_binding_streams import Fake


class Empty(Fake):
    def data_ptr(self):
        return 0


@pytest.fixture
def launched(monkeypatch):
    done = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: done.append(name) or 0
    monkeypatch.setattr(kv, "_lib", Lib())
    monkeypatch.setattr(kv, "_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda dev: 0)
    return done


class Rows(Fake):
    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)


LAY = kv.Layout(2, 64, 16)
U8, I32, F32, BF = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def pool():
    return Fake((5, 2, 16, 32), U8), Fake((5, 2, 16, 4), U8)


def append(**kw):
    r = Rows((3, 2, 64), BF)
    kv.nvfp4_kv_append(LAY, r, r, Fake((3,), torch.int64), *pool(), *pool(), **kw)


def bounds(**kw):
    kv.nvfp4_kv_page_bounds(LAY, *pool(), Fake((5, 2, 2, 64), torch.int8), Fake((5, 2), F32), **kw)


def select(**kw):
    kv.nvfp4_kv_select_pages(LAY, Fake((3, 4, 64), BF), Fake((5, 2, 2, 64), torch.int8), Fake((5, 2), F32), Fake((3, 9), I32),
                             Fake((3,), I32), Fake((3, 2, 4), I32), Fake((3, 2), I32), **kw)


def attend(k=None, v=None, **kw):
    one, q = Fake((1,), F32), Fake((3, 4, 64), BF)
    kv.nvfp4_paged_sparse_decode_attention(LAY, q, *pool(), k or one, *pool(), v or one, Fake((3, 2, 4), I32), Fake((3, 2), I32),
                                           0.1, q, workspace=Fake((1 << 20,), U8), **kw)


@pytest.mark.parametrize("call,name", [(append, "k_global_scale"), (append, "v_global_scale"), (append, "status"), (bounds, "status"),
                                       (select, "status"), (attend, "status"), (attend, "k"), (attend, "v")])
def test_an_empty_scalar_is_refused(launched, call, name):
    call()
    dtype = I32 if name == "status" else F32
    call(**{name: Fake((1,), dtype)})
    assert len(launched) == 2
    with pytest.raises(ValueError, match="at least one value"):
        call(**{name: Empty((0,), dtype)})
    assert len(launched) == 2
