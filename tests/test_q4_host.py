"""The 4-bit cache calls refuse bad arguments on the host (no GPU needed: every
call below fails validation before anything is enqueued)."""
import ctypes
import os

import pytest

import sparse_decode_attention_step_b200 as saga

OK = 1 << 40      # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(saga.LIB_PATH):
        from sparse_decode_attention_step_b200 import build
        build.build()
    return saga.load()


def good_shape(**kw):
    a = dict(B=2, h_q=16, h_k=2, h_v=4, d=64, dtype=saga.SAGA_BF16, cap=4096)
    a.update(kw)
    return saga.shape(**a)


def cache(**kw):
    a = dict(k_codes=OK, k_scales=OK, v_codes=OK, v_scales=OK, k_g=None, v_g=None)
    a.update(kw)
    return saga.saga_q4_cache(**a)


def calls(lib):
    """Each entry point as f(shape, cache, **arguments) with valid defaults."""
    b = ctypes.byref

    def run(fn, names, s, c, o):
        v = [o.get(n, d) for n, d in names]
        return fn(b(s) if s is not None else None, b(c) if c is not None else None, *v,
                  o.get("ws", OK), o.get("n_ws", 1 << 40), None)
    table = {
        "append": (lib.saga_q4_append_kv, [("k_new", OK), ("v_new", OK), ("T", 1), ("n_new", None), ("l", OK)]),
        "read": (lib.saga_q4_read_kv, [("start", None), ("n", 8), ("l", OK), ("K", OK), ("V", OK)]),
        "dense": (lib.saga_q4_dense_decode, [("q", OK), ("l", OK), ("out", OK)]),
        "step": (lib.saga_q4_decode_step, [("q", OK), ("l", OK), ("tau", OK), ("out", OK), ("cnt", None),
                                           ("mask", None)]),
        "refresh": (lib.saga_q4_refresh_threshold, [("q", OK), ("l", OK), ("N", 8), ("tau", OK), ("out", None),
                                                    ("cnt", None), ("mask", None), ("scores", None)]),
    }
    return {k: (lambda s, c, _f=f, _n=n, **o: run(_f, _n, s, c, o)) for k, (f, n) in table.items()}


NAMES = ["append", "read", "dense", "step", "refresh"]


@pytest.mark.parametrize("name", NAMES)
def test_shapes_refused(lib, name):
    call = calls(lib)[name]
    assert call(None, cache()) == saga.SAGA_ERR_INVALID_ARG
    assert call(good_shape(B=0), cache()) == saga.SAGA_ERR_INVALID_ARG
    assert call(good_shape(d=96), cache()) == saga.SAGA_ERR_UNSUPPORTED
    assert call(good_shape(cap=4098), cache()) == saga.SAGA_ERR_UNSUPPORTED       # cap % 4
    s = good_shape()
    s.v_stride_h += 64                                     # a multiple of 16 bytes, not of 256 values
    assert call(s, cache()) == saga.SAGA_ERR_UNSUPPORTED
    assert saga.q4_workspace_size(s) == 0
    assert call(good_shape(B=30000), cache()) == saga.SAGA_ERR_UNSUPPORTED        # B (h_k + h_v) > 65535


@pytest.mark.parametrize("name", NAMES)
def test_cache_pointers_refused(lib, name):
    call, s = calls(lib)[name], good_shape()
    assert call(s, None) == saga.SAGA_ERR_INVALID_ARG
    for f in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert call(s, cache(**{f: None})) == saga.SAGA_ERR_INVALID_ARG
        assert call(s, cache(**{f: OK + 8})) == saga.SAGA_ERR_INVALID_ARG
    assert call(s, cache(k_g=OK + 2)) == saga.SAGA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", NAMES)
def test_workspace_refused(lib, name):
    call, s = calls(lib)[name], good_shape()
    need = 256 if name in ("append", "read") else saga.q4_workspace_size(s)
    assert need % 256 == 0 and need > 0
    assert call(s, cache(), ws=None) == saga.SAGA_ERR_WORKSPACE
    assert call(s, cache(), ws=OK + 128) == saga.SAGA_ERR_WORKSPACE
    assert call(s, cache(), n_ws=need - 1) == saga.SAGA_ERR_WORKSPACE


@pytest.mark.parametrize("name,bad", [
    ("append", dict(k_new=None)), ("append", dict(v_new=OK + 8)), ("append", dict(T=0)),
    ("append", dict(l=None)), ("append", dict(n_new=OK + 2)),
    ("read", dict(n=0)), ("read", dict(K=None)), ("read", dict(V=OK + 4)), ("read", dict(l=OK + 1)),
    ("read", dict(start=OK + 2)),
    ("dense", dict(q=None)), ("dense", dict(q=OK + 8)), ("dense", dict(out=None)), ("dense", dict(out=OK + 8)),
    ("step", dict(tau=None)), ("step", dict(out=None)), ("step", dict(cnt=OK + 1)), ("step", dict(l=None)),
    ("refresh", dict(N=0)), ("refresh", dict(tau=None)), ("refresh", dict(out=OK + 8)),
    ("refresh", dict(cnt=OK)), ("refresh", dict(mask=OK)), ("refresh", dict(scores=OK + 2)),
])
def test_arguments_refused(lib, name, bad):
    assert calls(lib)[name](good_shape(), cache(), **bad) == saga.SAGA_ERR_INVALID_ARG


@pytest.mark.parametrize("hq,hk,hv,ok", [(16, 2, 16, False), (20, 2, 4, False), (32, 2, 8, True), (16, 1, 1, True)])
def test_dense_head_layouts(lib, hq, hk, hv, ok):
    s = good_shape(h_q=hq, h_k=hk, h_v=hv)
    # a supported layout gets as far as the workspace check
    want = saga.SAGA_ERR_WORKSPACE if ok else saga.SAGA_ERR_UNSUPPORTED
    assert calls(lib)["dense"](s, cache(), ws=None) == want
    assert calls(lib)["step"](s, cache(), ws=None) == saga.SAGA_ERR_WORKSPACE


@pytest.mark.parametrize("name", NAMES)
def test_longest_rows(lib, name):
    n = 2 ** 31 - 4096
    call = calls(lib)[name]
    assert call(good_shape(B=1, cap=n), cache(), ws=None) == saga.SAGA_ERR_UNSUPPORTED
    assert call(saga.shape(1, 16, 2, 4, 64, saga.SAGA_BF16, n, max_l_kv=n - 1), cache(), ws=None) == \
        saga.SAGA_ERR_WORKSPACE
