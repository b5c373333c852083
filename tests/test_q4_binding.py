"""What the Python binding of the 4-bit cache looks at before it hands addresses to
the library (no GPU needed: nothing is launched)."""
import os

import pytest
import torch

import sparse_decode_attention_step_b200 as saga

OK = 1 << 40      # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(saga.LIB_PATH):
        from sparse_decode_attention_step_b200 import build
        build.build()
    saga.load()


class Fake:
    """Stands in for a tensor of a GPU that is not there."""

    def __init__(self, shape, stride=None, dtype=torch.uint8, device="cuda:0"):
        t = torch.empty(shape, device="meta")
        self.shape, self.dtype, self.device = t.shape, dtype, torch.device(device)
        self._stride = t.stride() if stride is None else stride

    def stride(self):
        return self._stride

    def data_ptr(self):
        return OK


B, H_Q, H_K, H_V, D, CAP = 2, 16, 2, 4, 64, 512


def make(**kw):
    shp = saga.shape(B, H_Q, H_K, H_V, D, saga.SAGA_BF16, CAP)
    a = dict(k_codes=Fake((B, H_K, CAP, 32)), k_scales=Fake((B, H_K, CAP, 4)),
             v_codes=Fake((B, H_V, CAP, 32)), v_scales=Fake((B, H_V, CAP, 4)))
    a.update(kw)
    return shp, saga.Q4Cache(shp, **a)


def test_given_arrays_and_addresses():
    assert make()[1].c.k_codes == OK
    _, c = make(k_g=Fake((H_K,), dtype=torch.float32), v_g=Fake((H_V,), dtype=torch.float32))
    assert c.device == 0 and c.c.v_g == OK
    shp = saga.shape(B, H_Q, H_K, H_V, D, saga.SAGA_BF16, CAP)
    c = saga.Q4Cache(shp, OK, OK + 16, OK + 32, OK + 48, k_g=OK + 64)
    assert c.device is None and c.c.v_scales == OK + 48 and c.c.v_g is None
    # one sequence: its stride is never used
    one = saga.shape(1, H_Q, H_K, H_V, D, saga.SAGA_BF16, CAP)
    saga.Q4Cache(one, Fake((1, H_K, CAP, 32), (7, CAP * 32, 32, 1)), OK, OK, OK)


@pytest.mark.parametrize("bad", [
    dict(k_codes=Fake((B, H_K, CAP, 64))),                                  # 8 bits a value
    dict(k_codes=Fake((B, H_K, CAP, 32), dtype=torch.int8)),
    dict(k_scales=Fake((B, H_K, CAP, 4), dtype=torch.float32)),
    dict(v_codes=Fake((B, H_K, CAP, 32))),                                  # the key heads' size
    dict(v_codes=Fake((B, H_V, CAP, 32), (CAP * H_V * 32, 32, H_V * 32, 1))),   # heads inside positions
    dict(v_scales=Fake((B, H_V, CAP - 4, 4))),
    dict(v_scales=Fake((B * H_V * CAP * 4,))),
    dict(k_g=Fake((H_K,), dtype=torch.float64)),
    dict(k_g=Fake((H_K, 1), dtype=torch.float32)),
    dict(v_g=Fake((H_V,), (2,), dtype=torch.float32)),
    dict(v_g=Fake((H_K,), dtype=torch.float32)),
])
def test_arrays_of_another_type_size_or_layout_are_refused(bad):
    with pytest.raises(saga.SagaError) as e:
        make(**bad)
    assert e.value.status == saga.SAGA_ERR_INVALID_ARG and next(iter(bad)) in str(e.value)


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", ["k_codes", "k_scales", "v_codes", "v_scales", "k_g", "v_g"])
def test_arrays_of_two_devices_are_refused(name, device):
    h = H_K if name[0] == "k" else H_V
    x = (Fake((h,), dtype=torch.float32, device=device) if name.endswith("_g")
         else Fake((B, h, CAP, 32 if name.endswith("codes") else 4), device=device))
    with pytest.raises(saga.SagaError) as e:
        make(**{name: x})
    assert e.value.status == saga.SAGA_ERR_INVALID_ARG


def test_a_cache_or_workspace_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    shp, c = make()
    ws = Fake((1 << 20,))
    ws.nbytes, ws.device = 1 << 30, 1
    call = lambda c: saga.q4_dense_decode(shp, c, OK, OK, OK, ws, stream=0)
    with pytest.raises(saga.SagaError, match="a cache that is not on the current device"):
        call(c)
    here = saga.Q4Cache(shp, OK, OK, OK, OK)
    ws.device = 0
    with pytest.raises(saga.SagaError, match="a workspace that is not on the current device"):
        call(here)
