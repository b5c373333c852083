"""Python binding of the SAGA + Atop-N decode attention library (sm_100a).

A thin ctypes layer over ``include/saga.h`` (and ``saga_merge.h``, ``saga_q4.h``): the same entry points, the same
argument order, and argument marshalling only (device pointers from torch
tensors or plain integers, the CUDA stream handle). Every step of the
computation runs in the CUDA library ``_lib/libsaga_b200.so``; there is no
fallback, and every call fails loudly if the library is missing or returns an
error status.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# SAGA_CHECKED_BUILD=1 selects the bounds-checked build (build.py --check),
# SAGA_SHORT_WAITS_BUILD=1 the one whose 4-bit kernels give up their waits at once (--short-waits)
LIB_PATH = os.path.join(_HERE, "_lib", "libsaga_b200_check.so"
                        if os.environ.get("SAGA_CHECKED_BUILD") == "1" else "libsaga_b200_short.so"
                        if os.environ.get("SAGA_SHORT_WAITS_BUILD") == "1" else "libsaga_b200.so")

SAGA_OK = 0
SAGA_ERR_INVALID_ARG = 1
SAGA_ERR_UNSUPPORTED = 2
SAGA_ERR_WORKSPACE = 3
SAGA_ERR_CUDA = 4
SAGA_ERR_DEVICE = 5
SAGA_F32 = 0
SAGA_BF16 = 1
DEVERR_LKV_NEGATIVE = 1
DEVERR_LKV_TOO_LONG = 2


class SagaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = f"{where}: {status_string(status)} (status {status})"
        if status == SAGA_ERR_CUDA:
            msg += f": {last_error()}"
        super().__init__(msg)


class saga_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_k", ctypes.c_int32),
                ("h_v", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("cap", ctypes.c_int64), ("max_l_kv", ctypes.c_int64),
                ("q_stride_b", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
                ("v_stride_b", ctypes.c_int64), ("v_stride_h", ctypes.c_int64)]


class saga_merge_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("h_k", ctypes.c_int32), ("d", ctypes.c_int32)]


class saga_q4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("k_g", ctypes.c_void_p), ("v_g", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_SP = ctypes.POINTER(saga_shape)
_MP = ctypes.POINTER(saga_merge_shape)
_CP = ctypes.POINTER(saga_q4_cache)

_SIGS = {
    "saga_shape_contiguous": (None, [_SP, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_int64, ctypes.c_int64]),
    "saga_workspace_size": (ctypes.c_size_t, [_SP, ctypes.c_int32]),
    "saga_workspace_init": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "saga_decode_step": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        ctypes.c_size_t, _P]),
    "saga_refresh_threshold": (ctypes.c_int, [_SP, _P, _P, _P, _P, ctypes.c_int32, _P, _P,
                                              _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gqa_dense_decode": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "saga_dense_decode": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "saga_append_kv": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "saga_topn_step": (ctypes.c_int, [_SP, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "saga_debug_scores": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "saga_decode_step_noalloc": (ctypes.c_int, [_SP, _P, _P, _P, _P, _P, _P, _P, _P]),
    "saga_read_device_error": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "saga_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "saga_last_error": (ctypes.c_char_p, []),
    "saga_merge_workspace_size": (ctypes.c_size_t, [_MP]),
    "saga_merge_keys": (ctypes.c_int, [_MP, _P, _P, _P, ctypes.c_double, _P, _P, _P, _P, _P,
                                       ctypes.c_size_t, _P]),
    "saga_q4_workspace_size": (ctypes.c_size_t, [_SP]),
    "saga_q4_append_kv": (ctypes.c_int, [_SP, _CP, _P, _P, ctypes.c_int32, _P, _P, _P,
                                         ctypes.c_size_t, _P]),
    "saga_q4_read_kv": (ctypes.c_int, [_SP, _CP, _P, ctypes.c_int64, _P, _P, _P, _P,
                                       ctypes.c_size_t, _P]),
    "saga_q4_dense_decode": (ctypes.c_int, [_SP, _CP, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "saga_q4_decode_step": (ctypes.c_int, [_SP, _CP, _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_size_t, _P]),
    "saga_q4_refresh_threshold": (ctypes.c_int, [_SP, _CP, _P, _P, ctypes.c_int32, _P, _P, _P, _P,
                                                 _P, _P, ctypes.c_size_t, _P]),
}


def load():
    """Load the CUDA library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(
                f"{LIB_PATH} is missing: build it with "
                "`python sparse_decode_attention_step_b200/build.py`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc, where):
    if rc != SAGA_OK:
        raise SagaError(rc, where)


def status_string(status):
    return load().saga_status_string(status).decode()


def last_error():
    """The last CUDA failure a library call saw on this thread (or "")."""
    return load().saga_last_error().decode()


def shape(B, h_q, h_k, h_v, d, dtype, cap, max_l_kv=None):
    """A saga_shape for contiguous q [B][h_q][d], K [B][h_k][cap][d], V [B][h_v][cap][d]."""
    s = saga_shape()
    load().saga_shape_contiguous(ctypes.byref(s), B, h_q, h_k, h_v, d, dtype, cap,
                                 cap if max_l_kv is None else max_l_kv)
    return s


def workspace_size(shp, N=1):
    return int(load().saga_workspace_size(ctypes.byref(shp), N))


def workspace_init(ws, nbytes, stream=None):
    _check(load().saga_workspace_init(_ptr(ws), nbytes, _stream(stream)), "saga_workspace_init")


class Workspace:
    """Device workspace for one shape, allocated through torch and zeroed."""

    def __init__(self, shp, N=1, device="cuda", stream=None):
        import torch
        self.nbytes = workspace_size(shp, N)
        if self.nbytes == 0:
            raise SagaError(SAGA_ERR_INVALID_ARG, "saga_workspace_size")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        workspace_init(self.buf, self.nbytes, stream)

    def data_ptr(self):
        return self.buf.data_ptr()


def _ws(ws):
    return _ptr(ws), ws.nbytes


def decode_step(shp, q, K, V, l_kv, tau, out, ws, sel_count=None, sel_mask=None, stream=None):
    p, n = _ws(ws)
    _check(load().saga_decode_step(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V), _ptr(l_kv),
                                   _ptr(tau), _ptr(out), _ptr(sel_count), _ptr(sel_mask), p, n,
                                   _stream(stream)), "saga_decode_step")


def refresh_threshold(shp, q, K, l_kv, N, tau, ws, V=None, out=None, sel_count=None,
                      sel_mask=None, scores=None, stream=None):
    p, n = _ws(ws)
    _check(load().saga_refresh_threshold(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V),
                                         _ptr(l_kv), N, _ptr(tau), _ptr(out), _ptr(sel_count),
                                         _ptr(sel_mask), _ptr(scores), p, n, _stream(stream)),
           "saga_refresh_threshold")


def gqa_dense_decode(shp, q, K, V, l_kv, out, ws, stream=None):
    p, n = _ws(ws)
    _check(load().gqa_dense_decode(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V), _ptr(l_kv),
                                   _ptr(out), p, n, _stream(stream)), "gqa_dense_decode")


def dense_decode(shp, q, K, V, l_kv, out, ws, stream=None):
    """Full attention with the shape's key and value head maps (SAGA full
    attention when h_k < h_v, GQA full attention when h_k == h_v)."""
    p, n = _ws(ws)
    _check(load().saga_dense_decode(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V), _ptr(l_kv),
                                    _ptr(out), p, n, _stream(stream)), "saga_dense_decode")


def topn_step(shp, q, K, V, l_kv, N, out, ws, sel_count=None, sel_mask=None, scores=None,
              stream=None):
    """Exact top-N attention (ties to the lower position) for this step."""
    p, n = _ws(ws)
    _check(load().saga_topn_step(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V), _ptr(l_kv), N,
                                 _ptr(out), _ptr(sel_count), _ptr(sel_mask), _ptr(scores), p, n,
                                 _stream(stream)), "saga_topn_step")


def append_kv(shp, k_new, v_new, K, V, l_kv, ws, stream=None):
    """Write the token's key/value rows at position l_kv[b] and grow l_kv."""
    p, n = _ws(ws)
    _check(load().saga_append_kv(ctypes.byref(shp), _ptr(k_new), _ptr(v_new), _ptr(K), _ptr(V),
                                 _ptr(l_kv), p, n, _stream(stream)), "saga_append_kv")


NOALLOC_SCRATCH_BYTES = 160 << 20


def decode_step_noalloc(shp, q, K, V, l_kv, tau, out, sel_count=None, stream=None):
    """saga_decode_step with the library's fixed device scratch instead of a
    workspace, for callers that cannot allocate device memory."""
    _check(load().saga_decode_step_noalloc(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(V),
                                           _ptr(l_kv), _ptr(tau), _ptr(out), _ptr(sel_count),
                                           _stream(stream)), "saga_decode_step_noalloc")


def debug_scores(shp, q, K, l_kv, scores, ws, stream=None):
    p, n = _ws(ws)
    _check(load().saga_debug_scores(ctypes.byref(shp), _ptr(q), _ptr(K), _ptr(l_kv),
                                    _ptr(scores), p, n, _stream(stream)), "saga_debug_scores")


def read_device_error(ws, stream=None):
    """Synchronise, return and clear the device error word (0 = clean)."""
    flags = ctypes.c_int32(0)
    rc = load().saga_read_device_error(_ptr(ws), _stream(stream), ctypes.byref(flags))
    if rc not in (SAGA_OK, SAGA_ERR_DEVICE):
        raise SagaError(rc, "saga_read_device_error")
    return flags.value


# ---------------------------------------------------------------------------
# closed-form GQA-to-SAGA key-head merge (include/saga_merge.h)
# ---------------------------------------------------------------------------
def merge_shape(T, d_model, h_q, h_k, d):
    return saga_merge_shape(T, d_model, h_q, h_k, d)


def merge_workspace_size(mshape):
    return int(load().saga_merge_workspace_size(ctypes.byref(mshape)))


class MergeWorkspace:
    """Device workspace for saga_merge_keys, allocated through torch; its
    error word is zeroed."""

    def __init__(self, mshape, device="cuda", stream=None):
        import torch
        self.nbytes = merge_workspace_size(mshape)
        if self.nbytes == 0:
            raise SagaError(SAGA_ERR_INVALID_ARG, "saga_merge_workspace_size")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        workspace_init(self.buf, self.nbytes, stream)

    def data_ptr(self):
        return self.buf.data_ptr()


def merge_keys(mshape, X, W_K, Q, rcond, w, pairs, W_S, ws, total=None, stream=None):
    """Pair weights w [h_k][h_k] (float64), the minimum-weight pairing
    pairs [h_k/2][2] (int32) and the student's key projection
    W_S [h_k/2*d][d_model] (float32) from bf16 X [T][d_model],
    W_K [h_k*d][d_model] and Q [T][h_q*d]."""
    p, n = _ws(ws)
    _check(load().saga_merge_keys(ctypes.byref(mshape), _ptr(X), _ptr(W_K), _ptr(Q),
                                  float(rcond), _ptr(w), _ptr(pairs), _ptr(total), _ptr(W_S),
                                  p, n, _stream(stream)), "saga_merge_keys")


# ---------------------------------------------------------------------------
# the decode step over a KV cache held in 4 bits (include/saga_q4.h)
# ---------------------------------------------------------------------------
class Q4Cache:
    """The 4-bit caches of one shape: codes [B][h][cap][d/2] and scales
    [B][h][cap][d/16] (uint8) of K and V, and an optional fp32 scale per head
    (k_g [h_k], v_g [h_v]). Arrays not given are allocated through torch, with
    the shape's strides. A given tensor has to be on the GPU that the others are
    on, of its array's type and size and laid out by the shape's strides; a
    given address (an int) is taken as it is."""

    def __init__(self, shp, k_codes=None, k_scales=None, v_codes=None, v_scales=None, k_g=None,
                 v_g=None, device="cuda"):
        self.device = None

        def array(name, x, h, per, stride_b, stride_h):
            size = (shp.B, h, shp.cap, shp.d // per)
            strides = (stride_b // per, stride_h // per, shp.d // per, 1)
            if x is None:
                import torch
                n = sum((k - 1) * s for k, s in zip(size, strides)) + 1 if shp.cap > 0 else 0
                x = torch.zeros(n, dtype=torch.uint8, device=device).as_strided(size, strides)
            return self._given(name, x, "uint8", size, strides)
        self.k_codes = array("k_codes", k_codes, shp.h_k, 2, shp.k_stride_b, shp.k_stride_h)
        self.k_scales = array("k_scales", k_scales, shp.h_k, 16, shp.k_stride_b, shp.k_stride_h)
        self.v_codes = array("v_codes", v_codes, shp.h_v, 2, shp.v_stride_b, shp.v_stride_h)
        self.v_scales = array("v_scales", v_scales, shp.h_v, 16, shp.v_stride_b, shp.v_stride_h)
        self.k_g = self._given("k_g", k_g, "float32", (shp.h_k,), (1,))
        self.v_g = self._given("v_g", v_g, "float32", (shp.h_v,), (1,))
        self.c = saga_q4_cache(_ptr(self.k_codes), _ptr(self.k_scales), _ptr(self.v_codes),
                               _ptr(self.v_scales), _ptr(k_g), _ptr(v_g))

    def _given(self, name, x, dtype, size, strides):
        if x is None or isinstance(x, int):
            return x
        # the stride of a dimension of one entry is never used
        if (str(x.dtype) != "torch." + dtype or tuple(x.shape) != size or
                any(n > 1 and a != b for n, a, b in zip(size, x.stride(), strides))):
            raise SagaError(SAGA_ERR_INVALID_ARG, f"Q4Cache ({name}: {dtype} {list(size)} with strides "
                            f"{list(strides)} wanted, {x.dtype} {list(x.shape)} with {list(x.stride())} given)")
        if x.device.type != "cuda" or self.device not in (None, x.device.index):
            raise SagaError(SAGA_ERR_INVALID_ARG, f"Q4Cache ({name} is not on the GPU of the other arrays)")
        self.device = x.device.index
        return x


def q4_workspace_size(shp):
    return int(load().saga_q4_workspace_size(ctypes.byref(shp)))


class Q4Workspace:
    """Device workspace for the q4 calls of one shape, allocated through torch;
    its error word is zeroed. Calls that use it run on its device."""

    def __init__(self, shp, device="cuda", stream=None):
        import torch
        self.nbytes = q4_workspace_size(shp)
        if self.nbytes == 0:
            raise SagaError(SAGA_ERR_INVALID_ARG, "saga_q4_workspace_size")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.device = self.buf.device.index
        workspace_init(self.buf, self.nbytes, stream)

    def data_ptr(self):
        return self.buf.data_ptr()


def _q4(name, shp, cache, ws, stream, *args):
    """Call `name`(shape, cache, args..., workspace, stream). Arguments are ints,
    None or tensors; a tensor, the cache or the workspace on another device than
    the current one is refused (a kernel launched here could not reach it)."""
    import torch
    dev = torch.cuda.current_device()
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    v = []
    for x in args:
        if isinstance(x, torch.Tensor):
            if x.device.index != dev:
                raise SagaError(SAGA_ERR_INVALID_ARG, name + " (a tensor that is not on the current device)")
            x = x.data_ptr()
        v.append(x)
    if cache.device not in (None, dev):
        raise SagaError(SAGA_ERR_INVALID_ARG, name + " (a cache that is not on the current device)")
    if getattr(ws, "device", dev) != dev:
        raise SagaError(SAGA_ERR_INVALID_ARG, name + " (a workspace that is not on the current device)")
    rc = getattr(_lib or load(), name)(shp, cache.c, *v, ws.data_ptr(), ws.nbytes, stream)
    if rc != SAGA_OK:
        raise SagaError(rc, name)


def q4_append_kv(shp, cache, k_new, v_new, T, l_kv, ws, n_new=None, stream=None):
    """Quantise T new rows per sequence (n_new[b] of them where given), k_new
    [B][T][h_k][d] and v_new [B][T][h_v][d], write them at position l_kv[b]
    and grow l_kv."""
    _q4("saga_q4_append_kv", shp, cache, ws, stream, k_new, v_new, T, n_new, l_kv)


def q4_read_kv(shp, cache, n, l_kv, K, V, ws, start=None, stream=None):
    """Rows start[b] .. start[b] + n - 1 of every head into K [B][h_k][n][d] and
    V [B][h_v][n][d]; rows at or behind l_kv[b] are left as they were."""
    _q4("saga_q4_read_kv", shp, cache, ws, stream, start, n, l_kv, K, V)


def q4_dense_decode(shp, cache, q, l_kv, out, ws, stream=None):
    """Full attention over a 4-bit cache, with the shape's key and value head maps."""
    _q4("saga_q4_dense_decode", shp, cache, ws, stream, q, l_kv, out)


def q4_decode_step(shp, cache, q, l_kv, tau, out, ws, sel_count=None, sel_mask=None, stream=None):
    """One Atop-N step with stored thresholds over a 4-bit cache."""
    _q4("saga_q4_decode_step", shp, cache, ws, stream, q, l_kv, tau, out, sel_count, sel_mask)


def q4_refresh_threshold(shp, cache, q, l_kv, N, tau, ws, out=None, sel_count=None, sel_mask=None,
                         scores=None, stream=None):
    """Exact N-th largest scores over a 4-bit cache into tau; with out, the step too."""
    _q4("saga_q4_refresh_threshold", shp, cache, ws, stream, q, l_kv, N, tau, out, sel_count,
        sel_mask, scores)
