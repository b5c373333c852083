"""The 4-bit cache at the ends of its range: head scales and queries of any
magnitude, probabilities far under the largest, negative zeros, other orders of the
cache's dimensions, and the bounds-checked build."""
import os
import subprocess
import sys

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


@pytest.mark.parametrize("g", [2.0 ** 120, 2.0 ** -149])
@pytest.mark.parametrize("heads,d,cap", [((8, 2, 2), 64, 300), ((8, 2, 2), 64, 8200), ((12, 1, 4), 128, 8200)])
def test_value_heads_of_any_scale(heads, d, cap, g):
    """v_g at the ends of the range, in rows of one CTA and in rows that several share."""
    P = Problem(2, *heads, d, saga.SAGA_BF16, cap, [cap - 3, 0], 65, gscale=True)
    # blocks of scale 2^-6 for the large g and of 2^8 for the small one: values the type holds
    P.cache.v_scales.fill_(0x08 if g > 1 else 0x78)
    P.cache.v_g.fill_(g)
    P.V = q4.values(P.cache.v_codes.cpu().numpy(), P.cache.v_scales.cpu().numpy(), np.float32(g))
    tau = torch.full((2, heads[0]), -np.inf, device="cuda")
    cuda = lambda x: x.double().cpu().numpy()
    for call in (lambda: saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws),
                 lambda: saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws)):
        call()
        if g > 1:
            P.check_all(P.out)
            continue
        # outputs of few bits: half a step of 2^-149 and the bound's share of the largest value
        assert not P.out[1].any()
        for j in range(heads[0]):
            A = P.scores(0, j)
            p = np.exp(A - A.max())
            V = P.V[0, j * heads[2] // heads[0], :cap - 3]
            want = p @ V / p.sum()
            assert np.all(np.abs(cuda(P.out)[0, j] - want) <= 2.0 ** -149 + 1e-4 * np.abs(V).max())


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("g", [2.0 ** 120, 1.25 * 2.0 ** 120, 2.0 ** -149])
def test_read_back_of_any_head_scale(g, dtype):
    P = Problem(2, 8, 2, 4, 64, dtype, 300, [300, 41], 66, gscale=True)
    for codes, scales in ((P.cache.k_codes, P.cache.k_scales), (P.cache.v_codes, P.cache.v_scales)):
        codes[:, :, 7:9] = 0
        scales.fill_(0x08 if g > 1 else 0x78)
    P.cache.k_g.fill_(g)
    P.cache.v_g.fill_(g)
    tt = torch.float32 if dtype == saga.SAGA_F32 else torch.bfloat16
    K, V = torch.zeros(2, 2, 300, 64, dtype=tt, device="cuda"), torch.zeros(2, 4, 300, 64, dtype=tt, device="cuda")
    saga.q4_read_kv(P.shp, P.cache, 300, P.l, K, V, P.ws)
    for got, codes, scales in ((K, P.cache.k_codes, P.cache.k_scales), (V, P.cache.v_codes, P.cache.v_scales)):
        want = q4.values(codes.cpu().numpy(), scales.cpu().numpy(), np.float32(g)).astype(np.float32)
        for b, n in enumerate((300, 41)):
            assert torch.equal(got[b, :, :n].cpu(), torch.from_numpy(want[b, :, :n]).to(tt))


# ---------------------------------------------------------------------------
# probabilities far under the largest
# ---------------------------------------------------------------------------
# Keys of two kinds: "high" ones, of score s and value 0, and "low" ones, of
# score 0 and value 1, so that out = n w / (m + n w) with w = e^-s, m high and n low
# keys, in every element. Relative error of out: that of w (the product's factor has
# four roundings and the product one, each 2^-24 of the exponent s; the exponent's
# own rounding 2^-20 for an argument under 2^5 in log2 units, 2^-19 in two parts; ex2
# 2^-22, twice where it is taken in two parts), P's two halves (2^-22), the tensor cores'
# sums over at most 128 positions (2 units of 2^-23 in each of 16 steps for two
# halves), 2^-24 of every addition over a warp's chunks, and 2^-21 for the merges and
# the quotient.
def rel_bound(s, adds):
    return 5 * 2.0 ** -24 * s + 2.0 ** -20 + 2.0 ** -19 + 3 * 2.0 ** -22 + 16 * 2.0 ** -22 + 2 * adds * 2.0 ** -24 + 2.0 ** -21


def two_kinds(heads, d, B, L, high, weight, dtype):
    """(shape, cache, q, lengths, workspace, score s, expected output): `high` [L] bool, `weight` of a low key."""
    h_q, h_k, h_v = heads
    shp = saga.shape(B, h_q, h_k, h_v, d, dtype, L)
    g = np.float32(-np.log(weight) * np.sqrt(d) / 4)
    cache = saga.Q4Cache(shp, k_g=torch.full((h_k,), float(g), device="cuda"))
    cache.k_scales.fill_(0x38)
    cache.v_scales.fill_(0x38)
    cache.k_codes[:, :, high, 0] = 0x06                    # 4, then zeros
    cache.v_codes[:, :, ~high] = 0x22                      # ones
    q = torch.zeros(B, h_q, d, device="cuda", dtype=torch.float32 if dtype == saga.SAGA_F32 else torch.bfloat16)
    q[:, :, 0] = 1
    s = float(g) * 4 / np.sqrt(d)
    m, n, w = int(high.sum()), int((~high).sum()), np.exp(-s)
    l = torch.full((B,), L, dtype=torch.int32, device="cuda")
    return shp, cache, q, l, saga.Q4Workspace(shp), s, n * w / (m + n * w)


# every arrangement of score rows, with the sequences that give each CTA several chunks
LAYOUTS = [((8, 8, 8), 16), ((8, 1, 1), 64), ((16, 1, 1), 64), ((4, 1, 2), 64), ((16, 1, 2), 64), ((12, 1, 4), 64)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,B", LAYOUTS)
@pytest.mark.parametrize("bits", [14, 20, 24])
def test_dense_keeps_small_weights(bits, heads, B, d):
    """A few dominating keys at the head of each row, of value 0: what the others carry stays."""
    L = 16384
    t = torch.arange(L, device="cuda")
    shp, cache, q, l, ws, s, want = two_kinds(heads, d, B, L, (t < 1024) & (t % 32 == 0), 1.2345678 * 2.0 ** -bits,
                                              saga.SAGA_BF16)
    out = torch.zeros(B, heads[0], d, device="cuda")
    saga.q4_dense_decode(shp, cache, q, l, out, ws)
    err = (out.double() / want - 1).abs().max().item()
    assert err <= rel_bound(s, L // 128), (err, rel_bound(s, L // 128))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [14, 20, 24])
def test_step_keeps_small_weights(bits, d):
    """The same for the gather: each of its warps meets dominating keys first, then others."""
    L, heads, B = 8192, (12, 1, 4), 16
    t = torch.arange(L, device="cuda")
    shp, cache, q, l, ws, s, want = two_kinds(heads, d, B, L, t % 256 == 0, 1.2345678 * 2.0 ** -bits, saga.SAGA_BF16)
    out = torch.zeros(B, heads[0], d, device="cuda")
    saga.q4_decode_step(shp, cache, q, l, torch.full((B, heads[0]), -np.inf, device="cuda"), out, ws)
    err = (out.double() / want - 1).abs().max().item()
    assert err <= rel_bound(s, L // 32), (err, rel_bound(s, L // 32))


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,B", LAYOUTS)
@pytest.mark.parametrize("bits", [1, 6, 12])
def test_probabilities_have_their_low_halves(bits, heads, B, d, dtype):
    """High and low keys in turn: one fp16 half alone would be off by 1.6e-4 here."""
    L, B = 1024, 2
    shp, cache, q, l, ws, s, want = two_kinds(heads, d, B, L, torch.arange(L, device="cuda") % 2 == 0,
                                              1.2345678 * 2.0 ** -bits, dtype)
    tau = torch.full((B, heads[0]), -np.inf, device="cuda")
    for call in (lambda o: saga.q4_dense_decode(shp, cache, q, l, o, ws),
                 lambda o: saga.q4_decode_step(shp, cache, q, l, tau, o, ws)):
        out = torch.zeros(B, heads[0], d, device="cuda")
        call(out)
        err = (out.double() / want - 1).abs().max().item()
        assert err <= rel_bound(s, L // 32), (err, rel_bound(s, L // 32))


# ---------------------------------------------------------------------------
# negative zeros
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("T", [1, 3, 700])
def test_append_keeps_the_sign_of_zero(T, dtype):
    """-0 (and a quotient that rounds to it) among other values has the definition's code, 8."""
    rng = np.random.default_rng(67)
    shp = saga.shape(2, 4, 2, 4, 64, dtype, 704)
    x = {k: rng.standard_normal((2, T, h, 64)) for k, h in (("k", 2), ("v", 4))}
    for a in x.values():
        r = rng.random(a.shape)
        a[r < 0.2] = -0.0
        a[(r >= 0.2) & (r < 0.3)] = 0.0
        a[(r >= 0.3) & (r < 0.4)] = -1e-38
    x = {k: stored(a, dtype) for k, a in x.items()}
    cache, ws = saga.Q4Cache(shp), saga.Q4Workspace(shp)
    l = torch.zeros(2, dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, dev(x["k"], dtype), dev(x["v"], dtype), T, l, ws)
    for kind, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        wc, wsc = q4.quantise(x[kind].numpy())
        assert (wc & 15 == 8).any()
        assert np.array_equal(codes.cpu().numpy()[:, :, :T], wc.transpose(0, 2, 1, 3))
        assert np.array_equal(scales.cpu().numpy()[:, :, :T], wsc.transpose(0, 2, 1, 3))


# ---------------------------------------------------------------------------
# other orders of the cache's dimensions
# ---------------------------------------------------------------------------
def test_caches_with_the_heads_outermost():
    """[h][B][cap][d] caches, allocated by Q4Cache and written by append, against the usual order."""
    got = []
    for outer in (False, True):
        gen = torch.Generator("cuda").manual_seed(68)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()
        shp = saga.shape(3, 16, 2, 4, 64, saga.SAGA_BF16, 512)
        if outer:
            shp.k_stride_b = shp.v_stride_b = 512 * 64
            shp.k_stride_h = shp.v_stride_h = 3 * 512 * 64
        cache, ws = saga.Q4Cache(shp), saga.Q4Workspace(shp)
        l = torch.zeros(3, dtype=torch.int32, device="cuda")
        n = torch.tensor([512, 0, 77], dtype=torch.int32, device="cuda")
        saga.q4_append_kv(shp, cache, rand(3, 512, 2, 64), rand(3, 512, 4, 64), 512, l, ws, n_new=n)
        q, out, tau = rand(3, 16, 64), torch.zeros(3, 16, 64, device="cuda"), torch.zeros(3, 16, device="cuda")
        saga.q4_dense_decode(shp, cache, q, l, out, ws)
        dense = out.clone()
        saga.q4_refresh_threshold(shp, cache, q, l, 20, tau, ws, out=out)
        assert saga.read_device_error(ws) == 0
        got.append((cache.k_codes.clone(), cache.v_scales.clone(), dense, out, tau))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][2][0].any()


# ---------------------------------------------------------------------------
# the bounds-checked build over every kernel variant: the same bits, no check fails
# ---------------------------------------------------------------------------
CHAIN = r"""
import sys
import numpy as np, torch
import sparse_decode_attention_step_b200 as saga
saga.load()
res = {}
# every arrangement of score rows; rows of one position, of partial blocks and chunks, and
# too long for the select's chip; ties; windows that begin and end inside a row
for n, (d, heads, cap, lens, N, dt) in enumerate((
        (64, (8, 8, 8), 9000, (8997, 0, 1, 6401), 50, 1), (128, (8, 1, 1), 1300, (1, 1299, 33, 257), 1300, 1),
        (64, (16, 1, 1), 40000, (40000, 31, 32, 6145), 9000, 0), (128, (16, 1, 1), 9000, (8191, 2, 9000, 64), 3000, 0),
        (64, (4, 1, 2), 2000, (2000, 1024, 1, 0), 7, 1), (128, (16, 1, 2), 2000, (1999, 3, 640, 641), 300, 0),
        (64, (32, 2, 8), 150000, (149999, 0, 7, 512), 2048, 1), (128, (12, 1, 4), 9000, (9000, 5, 192, 193), 1, 1))):
    B, tt = len(lens), torch.bfloat16 if dt else torch.float32
    gen = torch.Generator("cuda").manual_seed(n)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(tt)
    shp = saga.shape(B, *heads, d, saga.SAGA_BF16 if dt else saga.SAGA_F32, cap)
    cache, ws = saga.Q4Cache(shp), saga.Q4Workspace(shp)
    l = torch.zeros(B, dtype=torch.int32, device="cuda")
    T = max(lens) - 1
    first = torch.tensor([max(x - 1, 0) for x in lens], dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, rand(B, T, heads[1], d), rand(B, T, heads[2], d), T, l, ws, n_new=first)
    last = torch.tensor([min(x, 1) for x in lens], dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, rand(B, 1, heads[1], d), rand(B, 1, heads[2], d), 1, l, ws, n_new=last)
    assert l.tolist() == list(lens)
    cache.k_codes[0, :, 100:600] = cache.k_codes[0, :, :1]       # ties
    cache.k_scales[0, :, 100:600] = cache.k_scales[0, :, :1]
    K = torch.zeros(B, heads[1], 301, d, device="cuda", dtype=tt)
    V = torch.zeros(B, heads[2], 301, d, device="cuda", dtype=tt)
    saga.q4_read_kv(shp, cache, 301, l, K, V, ws, start=(l - 200).clamp(min=0))
    q, out = rand(B, heads[0], d), torch.zeros(B, heads[0], d, device="cuda")
    tau, cnt = torch.zeros(B, heads[0], device="cuda"), torch.zeros(B, heads[0], dtype=torch.int32, device="cuda")
    mask = torch.zeros(B, heads[0], cap, dtype=torch.uint8, device="cuda")
    rows = torch.zeros(B, heads[0], cap, device="cuda")
    for k, call in enumerate((
            lambda: saga.q4_dense_decode(shp, cache, q, l, out, ws),
            lambda: saga.q4_refresh_threshold(shp, cache, q, l, N, tau, ws, out=out, sel_count=cnt, sel_mask=mask,
                                              scores=rows),
            lambda: saga.q4_refresh_threshold(shp, cache, q, l, max(1, N // 3), tau, ws),
            lambda: saga.q4_decode_step(shp, cache, q, l, tau, out, ws, sel_count=cnt, sel_mask=mask))):
        call()
        for name, x in (("out", out), ("tau", tau), ("cnt", cnt), ("mask", mask), ("rows", rows)):
            res[f"{n} {k} {name}"] = np.array([int(x.contiguous().view(torch.uint8).to(torch.int64).sum()),
                                               hash(x.cpu().numpy().tobytes())])
    res[f"{n} K"], res[f"{n} V"] = K.float().cpu().numpy(), V.float().cpu().numpy()
    res[f"{n} err"] = np.array([saga.read_device_error(ws)])
np.savez(sys.argv[1], **res)
"""


def test_checked_build_agrees_in_every_variant(tmp_path):
    from sparse_decode_attention_step_b200 import build
    if not os.path.exists(build.CHECK_LIB_PATH):
        build.build(check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = []
    for checked in ("0", "1"):
        path = str(tmp_path / f"{checked}.npz")
        env = dict(os.environ, SAGA_CHECKED_BUILD=checked, PYTHONHASHSEED="0",
                   PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
        r = subprocess.run([sys.executable, "-c", CHAIN, path], env=env, cwd=root, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(np.load(path))
    for k in got[0].files:
        assert np.array_equal(got[0][k], got[1][k]), k
        assert not k.endswith("err") or not got[1][k].any(), k
