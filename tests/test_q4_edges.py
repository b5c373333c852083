"""The 4-bit cache at the ends of its range: head scales and queries of any
magnitude, probabilities far under the largest, negative zeros."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_step_b200 as saga
from oracle import q4_cache as q4
from test_q4 import Problem, check_refresh, dev, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(gpu_lib):
    return gpu_lib


def rescale_keys(P, g, scale_byte=None):
    """Give every key head the scale g (and every block the scale byte), the codes as they are."""
    if scale_byte is not None:
        P.cache.k_scales.fill_(scale_byte)
    P.cache.k_g.fill_(g)
    P.K = q4.values(P.cache.k_codes.cpu().numpy(), P.cache.k_scales.cpu().numpy(), np.float32(g))


def set_queries(P, f):
    P.q.mul_(torch.tensor(f, device="cuda").view(1, -1, 1))
    P.q64 = P.q.double().cpu().numpy()


# ---------------------------------------------------------------------------
# products of a query's and a head's magnitude that leave the fp32 range
# ---------------------------------------------------------------------------
ROWS = [0.0, 1.0, 1e-30, 1e-38, 0.0, 1e-3, 1.0, 0.0]


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("heads,d", [((8, 2, 2), 64), ((8, 1, 1), 128), ((8, 1, 4), 64)])
@pytest.mark.parametrize("g", [1e-9, 2.0 ** -60, 2.0 ** -149])
def test_small_queries_times_small_head_scales(g, heads, d, dtype):
    """Scores that vanish weigh every position alike, and none behind the end."""
    P = Problem(4, *heads, d, dtype, 1300, [1299, 0, 1, 333], 61, gscale=True)
    rescale_keys(P, g)
    set_queries(P, ROWS)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    assert saga.read_device_error(P.ws) == 0
    P.check_all(P.out)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 50])
def test_refresh_of_zero_queries_and_small_head_scales(N, d, dtype):
    """Rows long enough for the bound from the group maxima, a partial block at their ends."""
    P = Problem(3, 8, 2, 4, d, dtype, 8200, [8197, 33, 6501], 62, gscale=True)
    rescale_keys(P, 1e-10)
    set_queries(P, [0.0, 1.0, 0.0, 1.0, 1.0, 0.0, 1.0, 0.0])
    check_refresh(P, N)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("heads,d", [((8, 2, 2), 64), ((12, 1, 4), 128)])
def test_small_queries_times_large_head_scales(heads, d, dtype):
    """k_g of 2^123 and queries of 2^-118: scores of ordinary size."""
    P = Problem(3, *heads, d, dtype, 8200, [8197, 0, 301], 63, gscale=True)
    rescale_keys(P, 2.0 ** 123, 0x08)                      # blocks of scale 2^-6
    set_queries(P, [2.0 ** -118] * heads[0])
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)
    check_refresh(P, 40)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
def test_zero_keys_times_large_queries(dtype):
    """Scores of zero whatever the factor: 0 times a factor past the fp32 range is not NaN."""
    P = Problem(2, 8, 2, 2, 64, dtype, 512, [512, 300], 64, gscale=True)
    P.cache.k_codes.zero_()
    rescale_keys(P, 2.0 ** 40)
    set_queries(P, [2.0 ** 100] * 8)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)
    check_refresh(P, 7)
