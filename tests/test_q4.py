"""The 4-bit cache on the GPU: quantised rows bit for bit, reading back, dense
decode, the Atop-N step and its refresh against float64 over the stored values.

Tolerances. A score is a sum of d exact products of fp16 operands in fp32 over
d/16 MMA steps (twice that for fp32 queries, whose low half adds as many); each
step loses at most 2 units of 2^-23 of the magnitudes added (S = sum |q k| /
sqrt(d)), the factors after it another 4: delta = 2 (steps + 4) 2^-23 S. An
fp32 query's own two halves keep 22 bits: one more 2^-22 S. A probability is
off by the scores of its key and of the maximum, by ex2 (2^-22), by its two fp16
halves (2^-22) and by the fp32 exponent's argument (2^-23 times its size, at
most the range R of the row's scores in log2 units plus 15); output sums lose
2 units of 2^-23 per 16 positions of one warp's share (at most 1/8 of a split
of 16384) and 64 more in the merges. So with e the sum of those,
|out - out*| <= 2 e sum_t p_t |v_t|, element by element."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as orc
import sparse_decode_attention_step_b200 as saga
from oracle import q4_cache as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(gpu_lib):
    return gpu_lib


JUNK = 0xFF        # what the caches hold where nothing was written


def stored(a, dtype):
    """fp32 values as the dtype stores them (still fp32)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t if dtype == saga.SAGA_F32 else t.to(torch.bfloat16).float()


def dev(t, dtype):
    return t.cuda() if dtype == saga.SAGA_F32 else t.to(torch.bfloat16).cuda()


def padded_shape(B, h_q, h_k, h_v, d, dtype, cap, max_l, pad):
    s = saga.shape(B, h_q, h_k, h_v, d, dtype, cap, max_l)
    if pad:
        s.q_stride_h += 16
        s.q_stride_b = h_q * s.q_stride_h + 32
        s.k_stride_h += 512
        s.k_stride_b = h_k * s.k_stride_h + 256
        s.v_stride_h += 256
        s.v_stride_b = h_v * s.v_stride_h + 768
    return s


def strided_q(shp, q, dtype):
    """q [B][h_q][d] with the shape's strides."""
    buf = torch.full((shp.B * shp.q_stride_b,), float("nan"), device="cuda",
                     dtype=torch.float32 if dtype == saga.SAGA_F32 else torch.bfloat16)
    v = buf.as_strided((shp.B, shp.h_q, shp.d), (shp.q_stride_b, shp.q_stride_h, 1))
    v.copy_(q)
    return v


class Problem:
    """A random cache of `lens` rows (junk behind them), its float64 values and queries."""

    def __init__(self, B, h_q, h_k, h_v, d, dtype, cap, lens, seed, pad=False, gscale=False, max_l=None,
                 planted=True):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.dtype, self.d, self.h_q, self.h_k, self.h_v, self.B = dtype, d, h_q, h_k, h_v, B
        self.shp = padded_shape(B, h_q, h_k, h_v, d, dtype, cap, cap if max_l is None else max_l, pad)
        self.gk = (rng.random(h_k).astype(np.float32) * 0.3 + 0.05) if gscale else np.ones(h_k, np.float32)
        self.gv = (rng.random(h_v).astype(np.float32) * 0.3 + 0.05) if gscale else np.ones(h_v, np.float32)
        K = rng.standard_normal((B, h_k, cap, d)).astype(np.float32)
        if planted:
            u = rng.standard_normal(d).astype(np.float32)
            hit = rng.random((B, h_k, cap)) < 0.02
            K[hit] = 3 * u / np.linalg.norm(u) + 0.5 * K[hit]
        V = rng.standard_normal((B, h_v, cap, d)).astype(np.float32)
        kc, ks = q4.quantise(K, self.gk[None, :, None, None])
        vc, vs = q4.quantise(V, self.gv[None, :, None, None])
        self.K = q4.values(kc, ks, self.gk[None, :, None, None])
        self.V = q4.values(vc, vs, self.gv[None, :, None, None])
        for b in range(B):
            for a in (kc, ks, vc, vs):
                a[b, :, self.lens[b]:] = JUNK
        dg = lambda g: torch.from_numpy(g).cuda() if gscale else None
        self.cache = saga.Q4Cache(self.shp, k_g=dg(self.gk), v_g=dg(self.gv))
        for t, a in ((self.cache.k_codes, kc), (self.cache.k_scales, ks), (self.cache.v_codes, vc),
                     (self.cache.v_scales, vs)):
            t.copy_(torch.from_numpy(a))
        q = stored(rng.standard_normal((B, h_q, d)), dtype)
        self.q64 = q.double().numpy()
        self.q = strided_q(self.shp, dev(q, dtype), dtype)
        self.l = torch.from_numpy(self.lens).cuda()
        self.ws = saga.Q4Workspace(self.shp)
        self.out = torch.full((B, h_q, d), float("nan"), device="cuda")

    def scores(self, b, j):
        kh = orc.key_head(j, self.h_q, self.h_k)
        return self.K[b, kh, :self.lens[b]] @ self.q64[b, j] / np.sqrt(self.d)

    def delta(self, b, j):
        kh = orc.key_head(j, self.h_q, self.h_k)
        S = np.max(np.abs(self.K[b, kh, :self.lens[b]]) @ np.abs(self.q64[b, j])) / np.sqrt(self.d)
        wide = self.dtype == saga.SAGA_F32
        return S * (2 * ((2 if wide else 1) * self.d / 16 + 4) * 2.0 ** -23 + (2.0 ** -22 if wide else 0))

    def check_out(self, out, b, j, sel=None):
        """out[b][j] against softmax attention over positions `sel` (all by default)."""
        A = self.scores(b, j)
        sel = np.arange(A.size) if sel is None else sel
        if sel.size == 0:
            assert not out.any()
            return
        Vr = self.V[b, orc.value_head(j, self.h_q, self.h_v), sel]
        p = np.exp(A[sel] - A[sel].max())
        p /= p.sum()
        R = (A[sel].max() - A[sel].min()) * 1.4427 + 15
        e = (2 * self.delta(b, j) + 2 * 2.0 ** -22 + 2.0 ** -23 * R
             + 2.0 ** -22 * (min(A.size, 2048) / 16 + 64))
        err = np.abs(out.astype(np.float64) - p @ Vr)
        assert np.all(err <= 2 * e * (p @ np.abs(Vr))), (b, j, np.max(err / (p @ np.abs(Vr))), 2 * e)

    def check_all(self, out, rows=None):
        out = out.cpu().numpy()
        for b in range(self.B):
            for j in range(self.h_q) if rows is None else rows:
                if self.lens[b] == 0:
                    assert not out[b, j].any()
                else:
                    self.check_out(out[b, j], b, j)


# ---------------------------------------------------------------------------
# append and read back
# ---------------------------------------------------------------------------
def append_case(B, h_k, h_v, d, dtype, cap, l0, T, n_new, gscale, pad, seed, special=False):
    rng = np.random.default_rng(seed)
    shp = padded_shape(B, h_v, h_k, h_v, d, dtype, cap, cap, pad)
    x = {"k": rng.standard_normal((B, T, h_k, d)) * np.exp2(rng.integers(-6, 7, (B, T, h_k, 1))),
         "v": rng.standard_normal((B, T, h_v, d))}
    if special:
        for a in x.values():
            a[rng.random(a.shape) < 0.01] = np.nan
            a[rng.random(a.shape) < 0.002] = np.inf
            a[rng.random(a.shape) < 0.002] = -np.inf
            a[rng.random(a.shape) < 0.05] = 0.0
            a[:, :, :, 16:32] *= 1e-6
            a[:, :, :, 32:48] = -0.0
    x = {k: stored(v, dtype) for k, v in x.items()}
    g = {"k": rng.random(h_k).astype(np.float32) * 0.3 + 0.05 if gscale else np.ones(h_k, np.float32),
         "v": rng.random(h_v).astype(np.float32) * 0.3 + 0.05 if gscale else np.ones(h_v, np.float32)}
    dg = lambda a: torch.from_numpy(a).cuda() if gscale else None
    cache = saga.Q4Cache(shp, k_g=dg(g["k"]), v_g=dg(g["v"]))
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(JUNK)
    l = torch.tensor(l0, dtype=torch.int32, device="cuda")
    ws = saga.Q4Workspace(shp)
    n = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, dev(x["k"], dtype), dev(x["v"], dtype), T, l, ws, n_new=n)
    torch.cuda.synchronize()
    return shp, x, g, cache, l, ws


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("B,h_k,h_v,d,cap,l0,T,n_new,gscale,pad", [
    (1, 1, 4, 128, 64, [5], 1, None, False, False),            # one token
    (3, 2, 4, 64, 1028, [0, 517, 1020], 1, None, True, True),  # a token of a ragged batch
    (4, 1, 2, 64, 128, [0, 3, 90, 128], 37, [37, 0, 36, 0], False, True),
    (2, 2, 2, 128, 2048, [1, 777], 613, [613, 300], True, False),
    (3, 2, 8, 64, 1500, [0, 0, 1], 1499, None, False, False),   # a prompt up to the last row
])
def test_append_is_the_quantiser_bit_for_bit(dtype, B, h_k, h_v, d, cap, l0, T, n_new, gscale, pad):
    shp, x, g, cache, l, ws = append_case(B, h_k, h_v, d, dtype, cap, l0, T, n_new, gscale, pad, 11 + T)
    n = [T] * B if n_new is None else n_new
    assert saga.read_device_error(ws) == 0
    assert l.tolist() == [a + b for a, b in zip(l0, n)]
    for kind, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        wc, wsc = q4.quantise(x[kind].numpy(), g[kind][None, None, :, None])
        gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
        for b in range(B):
            a, e = l0[b], l0[b] + n[b]
            assert np.array_equal(gc[b, :, a:e], wc[b, :n[b]].transpose(1, 0, 2)), (kind, b)
            assert np.array_equal(gs[b, :, a:e], wsc[b, :n[b]].transpose(1, 0, 2)), (kind, b)
            for got in (gc, gs):                       # nothing else was touched
                assert np.all(got[b, :, :a] == JUNK) and np.all(got[b, :, e:] == JUNK)


def test_append_special_values():
    shp, x, g, cache, l, ws = append_case(2, 1, 2, 64, saga.SAGA_F32, 256, [0, 7], 200, None, False, False, 5,
                                          special=True)
    for kind, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        wc, wsc = q4.quantise(x[kind].numpy())
        for b, a in enumerate([0, 7]):
            assert np.array_equal(codes.cpu().numpy()[b, :, a:a + 200], wc[b].transpose(1, 0, 2))
            assert np.array_equal(scales.cpu().numpy()[b, :, a:a + 200], wsc[b].transpose(1, 0, 2))


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("g_exp,x_exp", [(-105, 126), (-105, 0), (-120, -100), (100, 126), (120, 0), (0, -120)])
def test_append_far_from_the_scales_range(dtype, g_exp, x_exp):
    # quotients that overflow, scales that stop at 448 or vanish, t outside of the fast path
    shp = saga.shape(1, 2, 1, 2, 64, dtype, 64)
    rng = np.random.default_rng(9)
    x = {k: stored(rng.uniform(-1, 1, (1, 50, h, 64)) * 2.0 ** x_exp, dtype) for k, h in (("k", 1), ("v", 2))}
    g = {"k": np.full(1, 2.0 ** g_exp, np.float32), "v": np.full(2, 1.25 * 2.0 ** g_exp, np.float32)}
    cache = saga.Q4Cache(shp, k_g=torch.from_numpy(g["k"]).cuda(), v_g=torch.from_numpy(g["v"]).cuda())
    l = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = saga.Q4Workspace(shp)
    saga.q4_append_kv(shp, cache, dev(x["k"], dtype), dev(x["v"], dtype), 50, l, ws)
    assert saga.read_device_error(ws) == 0
    for kind, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        wc, wsc = q4.quantise(x[kind].numpy(), g[kind][None, None, :, None])
        assert np.array_equal(codes.cpu().numpy()[0, :, :50], wc[0].transpose(1, 0, 2))
        assert np.array_equal(scales.cpu().numpy()[0, :, :50], wsc[0].transpose(1, 0, 2))


@pytest.mark.parametrize("T", [1, 300])
def test_append_leaves_a_sequence_without_room(T):
    # full, negative length, n > T, n < 0, and one that fits to the last row
    l0, n = [512 - T + 1, -1, 0, 0, 512 - T], [T, T, T + 1, -1, T]
    shp, x, g, cache, l, ws = append_case(5, 2, 4, 64, saga.SAGA_BF16, 512, l0, T, n, False, False, 3)
    assert saga.read_device_error(ws) == saga.DEVERR_LKV_TOO_LONG | saga.DEVERR_LKV_NEGATIVE
    assert l.tolist() == l0[:4] + [512]
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert torch.all(t[:4] == JUNK) and torch.all(t[4, :, :512 - T] == JUNK)
        assert not torch.all(t[4, :, 512 - T:] == JUNK)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d,lens,start,n,gscale,pad", [
    (64, [1300, 0, 301], None, 1300, True, False),
    (128, [900, 64, 1], [899, 10, 0], 77, True, True),
    (64, [1027, 1300, 5], [1000, 1299, 5], 1, False, True),
    (128, [40, 1300, 1300], [-1, 1296, 1301], 4, False, False),
])
def test_read_is_exact_and_leaves_what_is_behind(dtype, d, lens, start, n, gscale, pad):
    P = Problem(3, 8, 2, 4, d, dtype, 1300, lens, 7, pad=pad, gscale=gscale)
    tt = torch.float32 if dtype == saga.SAGA_F32 else torch.bfloat16
    K = torch.full((3, 2, n, d), 77.0, dtype=tt, device="cuda")
    V = torch.full((3, 4, n, d), 77.0, dtype=tt, device="cuda")
    st = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    saga.q4_read_kv(P.shp, P.cache, n, P.l, K, V, P.ws, start=st)
    err = saga.read_device_error(P.ws)
    assert err == (saga.DEVERR_LKV_NEGATIVE if start is not None and min(start) < 0 else 0)
    for got, vals in ((K, P.K), (V, P.V)):
        want = torch.full(got.shape, 77.0)
        for b in range(3):
            a = 0 if start is None else start[b]
            e = min(a + n, lens[b])
            if a >= 0 and e > a:               # code * scale is exact, times g rounds once to fp32
                want[b, :, :e - a] = torch.from_numpy(vals[b, :, a:e].astype(np.float32))
        assert torch.equal(got.cpu(), want.to(tt))


# ---------------------------------------------------------------------------
# dense decode
# ---------------------------------------------------------------------------
LAYOUTS = [(8, 8, 8), (4, 1, 1), (12, 2, 2), (16, 2, 2), (9, 1, 1), (16, 1, 1),      # one value head
           (4, 1, 2), (12, 1, 2), (32, 2, 4), (16, 2, 4),                           # two
           (4, 1, 4), (12, 1, 4), (32, 2, 8), (16, 1, 4)]                           # four


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", LAYOUTS)
def test_dense_every_layout(heads, d, dtype):
    P = Problem(4, *heads, d, dtype, 1300, [1300, 0, 1, 301], 21, gscale=True)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    assert saga.read_device_error(P.ws) == 0
    P.check_all(P.out)


@pytest.mark.parametrize("heads,d", [((8, 2, 2), 64), ((12, 1, 4), 128)])
@pytest.mark.parametrize("lens", [[2, 3, 4, 5], [31, 32, 33, 63], [127, 128, 129, 130], [255, 256, 257, 258],
                                  [511, 513, 1023, 1025]])
def test_dense_lengths_and_strides(heads, d, lens):
    P = Problem(4, *heads, d, saga.SAGA_BF16, 1100, lens, 5, pad=True, max_l=1026)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)


@pytest.mark.parametrize("heads,d,dtype", [((8, 1, 1), 64, saga.SAGA_BF16), ((4, 1, 4), 128, saga.SAGA_F32)])
def test_dense_long(heads, d, dtype):
    P = Problem(1, *heads, d, dtype, 70004, [70001], 9)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)


def test_dense_rows_of_one_score_and_rising_scores():
    """Equal keys, and scores that rise along the row (every rescale of the running maximum)."""
    P = Problem(2, 8, 2, 2, 64, saga.SAGA_F32, 2048, [2048, 2048], 4)
    P.cache.k_codes[0].copy_(P.cache.k_codes[0, :, :1].expand_as(P.cache.k_codes[0]))
    P.cache.k_scales[0].copy_(P.cache.k_scales[0, :, :1].expand_as(P.cache.k_scales[0]))
    rise = torch.sort(P.cache.k_scales[1].view(torch.uint8).int() * 0 + (torch.arange(2048, device="cuda") // 18 + 8)[None, :, None], 1).values
    P.cache.k_codes[1].copy_(P.cache.k_codes[1, :, :1].expand_as(P.cache.k_codes[1]))
    P.cache.k_scales[1].copy_(rise.to(torch.uint8))
    P.K = q4.values(P.cache.k_codes.cpu().numpy(), P.cache.k_scales.cpu().numpy())
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)


def test_dense_query_magnitudes():
    """Queries from the smallest to large magnitudes, a zero row and a zero cache."""
    P = Problem(2, 8, 2, 2, 64, saga.SAGA_F32, 512, [512, 512], 6)
    f = torch.tensor([1e-30, 1e-3, 1.0, 3.0, 0.0, 1e-38, 1e-6, 0.5], device="cuda").view(1, 8, 1)
    P.q.mul_(f)
    P.q64 = P.q.double().cpu().numpy()
    P.cache.k_scales[1].zero_()
    P.K[1] = 0
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)


def test_lengths_out_of_range_are_clamped():
    P = Problem(3, 8, 2, 4, 64, saga.SAGA_BF16, 512, [512, 100, 300], 6)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    want = P.out.clone()
    l = torch.tensor([513, -3, 300], dtype=torch.int32, device="cuda")
    tau = torch.full((3, 8), -np.inf, device="cuda")
    for call in (lambda: saga.q4_dense_decode(P.shp, P.cache, P.q, l, P.out, P.ws),
                 lambda: saga.q4_decode_step(P.shp, P.cache, P.q, l, tau, P.out, P.ws)):
        call()
        assert saga.read_device_error(P.ws) == saga.DEVERR_LKV_TOO_LONG | saga.DEVERR_LKV_NEGATIVE
        torch.testing.assert_close(P.out[0], want[0], rtol=1e-4, atol=1e-5)
        assert not P.out[1].any()


# ---------------------------------------------------------------------------
# the Atop-N step and its refresh
# ---------------------------------------------------------------------------
def check_step(P, out, cnt, mask, tau, rows=None):
    out, cnt, mask, tau = out.cpu().numpy(), cnt.cpu().numpy(), mask.cpu().numpy(), tau.cpu().numpy()
    for b in range(P.B):
        L = int(P.lens[b])
        for j in range(P.h_q) if rows is None else rows:
            assert np.all(mask[b, j, L:] == 2), "mask entries beyond l_kv were written"
            assert np.all((mask[b, j, :L] == 0) | (mask[b, j, :L] == 1))
            sel = np.nonzero(mask[b, j, :L] == 1)[0]
            assert cnt[b, j] == sel.size
            if L == 0:
                assert not out[b, j].any()
                continue
            A = P.scores(b, j)
            diff = np.setxor1d(sel, np.nonzero(A >= float(tau[b, j]))[0])
            assert np.all(np.abs(A[diff] - tau[b, j]) <= P.delta(b, j)), (b, j, diff[:8])
            P.check_out(out[b, j], b, j, sel)


def run_step(P, tau):
    cnt = torch.zeros(P.B, P.h_q, dtype=torch.int32, device="cuda")
    mask = torch.full((P.B, P.h_q, P.shp.max_l_kv), 2, dtype=torch.uint8, device="cuda")
    saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws, sel_count=cnt, sel_mask=mask)
    assert saga.read_device_error(P.ws) == 0
    return cnt, mask


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4, 4), (6, 1, 3), (12, 1, 4), (16, 2, 16), (32, 2, 8), (9, 1, 1)])
def test_step_every_layout(heads, d, dtype):
    P = Problem(4, *heads, d, dtype, 1300, [1300, 0, 1, 301], 33, gscale=True, pad=True, max_l=1299 + 1)
    A = np.stack([np.sort(np.concatenate([P.scores(0, j), np.zeros(0)]))[-60] for j in range(P.h_q)])
    tau = torch.from_numpy(np.broadcast_to(A, (4, P.h_q)).astype(np.float32).copy()).cuda()
    tau[:, 0] = -np.inf                          # keeps everything
    tau[:, 1] = np.inf                           # keeps nothing
    cnt, mask = run_step(P, tau)
    check_step(P, P.out, cnt, mask, tau)
    assert cnt[:, 0].tolist() == P.lens.tolist() and not cnt[:, 1].any()
    got = P.out.clone()
    saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws)   # without counts and mask
    assert torch.equal(got, P.out)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("heads,d,cap,lens,N", [
    ((4, 1, 2), 64, 1024, [1024, 1000, 64], 64),
    ((32, 2, 8), 64, 1300, [1300, 0, 301], 40),
    ((12, 1, 4), 128, 5004, [5003, 40, 41], 40),
    ((16, 1, 1), 128, 300, [300, 299, 1], 1),
])
def test_refresh_and_step(heads, d, cap, lens, N, dtype):
    P = Problem(3, *heads, d, dtype, cap, lens, 17, gscale=True)
    B, h_q = P.B, P.h_q
    tau = torch.full((B, h_q), float("nan"), device="cuda")
    rows = torch.full((B, h_q, cap), 777.0, device="cuda")
    cnt = torch.zeros(B, h_q, dtype=torch.int32, device="cuda")
    mask = torch.full((B, h_q, cap), 2, dtype=torch.uint8, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt, sel_mask=mask,
                              scores=rows)
    assert saga.read_device_error(P.ws) == 0
    r, t = rows.cpu().numpy(), tau.cpu().numpy()
    for b in range(B):
        L = lens[b]
        for j in range(h_q):
            assert np.all(r[b, j, L:] == 777)
            want = orc.nth_largest_f32(r[b, j, :L], N)
            assert np.float32(want).view(np.uint32) == t[b, j].view(np.uint32), (b, j)
            if L:
                assert np.max(np.abs(r[b, j, :L] - P.scores(b, j))) <= P.delta(b, j)
            keep = r[b, j, :L] >= t[b, j]
            assert np.array_equal(mask[b, j, :L].cpu().numpy(), keep.astype(np.uint8))
    check_step(P, P.out, cnt, mask, tau)
    # tau alone, rows kept in the workspace: the same thresholds
    tau2 = torch.zeros_like(tau)
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau2, P.ws)
    assert torch.equal(tau, tau2)
    # and the step with the stored thresholds is the refresh's own
    cnt2, mask2 = run_step(P, tau)
    assert torch.equal(cnt, cnt2) and torch.equal(mask, mask2)


def test_step_long_rows():
    P = Problem(1, 16, 1, 4, 64, saga.SAGA_BF16, 70004, [70001], 8, gscale=True)
    tau = torch.full((1, 16), 0.0, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, 2048, tau, P.ws)
    cnt, mask = run_step(P, tau)
    assert cnt.tolist() == [[2048] * 16] or cnt.min() >= 2048
    check_step(P, P.out, cnt, mask, tau, rows=[0, 5, 15])


@pytest.mark.parametrize("N", [1, 40, 700])
def test_nan_and_infinite_queries_stay_in_their_rows(N):
    """A query row of NaN or infinities leaves its own outputs undefined, ends like
    any other, and changes no other row."""
    P = Problem(2, 16, 2, 4, 64, saga.SAGA_F32, 1300, [1300, 900], 19)
    tau = torch.zeros(2, 16, device="cuda")
    cnt = torch.zeros(2, 16, dtype=torch.int32, device="cuda")

    def run():
        saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt)
        a = (tau.clone(), P.out.clone(), cnt.clone())
        saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws, sel_count=cnt)
        b = (P.out.clone(), cnt.clone())
        saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
        return a + b + (P.out.clone(),)
    clean = run()
    P.q[0, 1, 3] = float("nan")
    P.q[0, 9, :] = float("nan")
    P.q[1, 2, 5] = float("inf")
    P.q[1, 14, :] = float("-inf")
    got = run()
    assert saga.read_device_error(P.ws) == 0
    ok = torch.ones(2, 16, dtype=torch.bool)
    for b, j in ((0, 1), (0, 9), (1, 2), (1, 14)):
        ok[b, j] = False
    for x, y in zip(got, clean):
        assert torch.equal(x.cpu()[ok], y.cpu()[ok])


@pytest.mark.parametrize("N", [1, 9000, 19999])
def test_refresh_of_rows_of_one_score(N):
    """Every score tied: each list holds the whole row, which is too long for the chip."""
    P = Problem(2, 8, 1, 2, 64, saga.SAGA_BF16, 20000, [20000, 12000], 23)
    for t in (P.cache.k_codes, P.cache.k_scales):
        t.copy_(t[:, :, :1].expand_as(t).clone())
    P.K[:] = P.K[:, :, :1]
    tau = torch.zeros(2, 8, device="cuda")
    cnt = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt)
    for b in range(2):
        assert cnt[b].tolist() == [int(P.lens[b])] * 8
        for j in range(8):
            if N >= P.lens[b]:
                assert tau[b, j] == -np.inf
            else:
                assert abs(float(tau[b, j]) - P.scores(b, j)[0]) <= P.delta(b, j)
    P.check_all(P.out)


@pytest.mark.parametrize("N", [3000, 9000, 15000])
def test_refresh_with_a_large_share_kept(N):
    """Lists that do not fit the chip, dense and sparse, against the sorted score rows."""
    P = Problem(2, 8, 1, 2, 64, saga.SAGA_BF16, 60000, [60000, 16001], 29)
    tau = torch.zeros(2, 8, device="cuda")
    rows = torch.zeros(2, 8, 60000, device="cuda")
    cnt = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    mask = torch.full((2, 8, 60000), 2, dtype=torch.uint8, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt, sel_mask=mask,
                              scores=rows)
    for b in range(2):
        L = int(P.lens[b])
        s = rows[b, :, :L].sort(-1, descending=True).values
        assert torch.equal(tau[b], s[:, N - 1])
        assert torch.equal(mask[b, :, :L], (rows[b, :, :L] >= tau[b, :, None]).to(torch.uint8))
        assert torch.all(mask[b, :, L:] == 2)
        assert torch.equal(cnt[b], (rows[b, :, :L] >= tau[b, :, None]).sum(-1, dtype=torch.int32))
    check_step(P, P.out, cnt, mask, tau, rows=[0, 7])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
def test_prompt_then_tokens(dtype):
    """Prompts of different lengths, then token by token: append, a refresh
    every third step, plain steps between, dense beside them; every step over the
    rows stored so far. The same tokens from a captured graph give the same bits."""
    B, h_q, h_k, h_v, d, cap, N, T = 3, 16, 2, 4, 64, 700, 24, 7
    rng = np.random.default_rng(40)
    P = Problem(B, h_q, h_k, h_v, d, dtype, cap, [0, 0, 0], 1)
    n0 = np.array([600, 0, 333], np.int32)
    k0, v0 = stored(rng.standard_normal((B, 600, h_k, d)), dtype), stored(rng.standard_normal((B, 600, h_v, d)), dtype)
    kt, vt = stored(rng.standard_normal((T, B, 1, h_k, d)), dtype), stored(rng.standard_normal((T, B, 1, h_v, d)), dtype)
    qt = stored(rng.standard_normal((T, B, h_q, d)), dtype)
    dk, dv = [dev(x, dtype) for x in kt], [dev(x, dtype) for x in vt]
    saga.q4_append_kv(P.shp, P.cache, dev(k0, dtype), dev(v0, dtype), 600, P.l, P.ws, n_new=torch.from_numpy(n0).cuda())
    for kind, vals in (("k", k0), ("v", v0)):
        c, s = q4.quantise(vals.numpy())
        v = q4.values(c, s).transpose(0, 2, 1, 3)
        (P.K if kind == "k" else P.V)[:, :, :600] = v
    tau = torch.zeros(B, h_q, device="cuda")
    cnt = torch.zeros(B, h_q, dtype=torch.int32, device="cuda")
    mask = torch.zeros(B, h_q, cap, dtype=torch.uint8, device="cuda")
    dense, q = torch.zeros_like(P.out), P.q

    def token(t):
        saga.q4_append_kv(P.shp, P.cache, dk[t], dv[t], 1, P.l, P.ws)
        mask.fill_(2)
        if t % 3 == 0:
            saga.q4_refresh_threshold(P.shp, P.cache, q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt, sel_mask=mask)
        else:
            saga.q4_decode_step(P.shp, P.cache, q, P.l, tau, P.out, P.ws, sel_count=cnt, sel_mask=mask)
        saga.q4_dense_decode(P.shp, P.cache, q, P.l, dense, P.ws)

    seen = []
    for t in range(T):
        q.copy_(dev(qt[t], dtype))
        P.q64 = qt[t].double().numpy()
        token(t)
        assert saga.read_device_error(P.ws) == 0
        P.lens = n0 + t + 1
        assert P.l.tolist() == P.lens.tolist()
        for vals, new in ((P.K, kt[t]), (P.V, vt[t])):
            c, s = q4.quantise(new.numpy())
            for b in range(B):
                vals[b, :, n0[b] + t] = q4.values(c, s)[b, 0]
        check_step(P, P.out, cnt, mask, tau)
        P.check_all(dense)
        seen.append((P.out.clone(), dense.clone(), tau.clone()))
    # the same from graphs, on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.l.copy_(torch.from_numpy(n0))
        tau.zero_()
        graphs = []
        for t in range(T):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                token(t)
            graphs.append(g)
        P.l.copy_(torch.from_numpy(n0))
        tau.zero_()
        for t in range(T):
            q.copy_(dev(qt[t], dtype))
            graphs[t].replay()
            side.synchronize()
            for got, want in zip((P.out, dense, tau), seen[t]):
                assert torch.equal(got, want), t
    torch.cuda.current_stream().wait_stream(side)


def test_two_streams_at_once():
    """Calls with their own workspaces on two streams at once give what they give alone."""
    Ps = [Problem(4, 16, 2, 4, 64, saga.SAGA_BF16, 2000, [2000, 1, 900, 1500], s) for s in (1, 2)]
    taus = [torch.full((4, 16), 1.5, device="cuda") for _ in Ps]

    def work(P, tau):
        saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
        a = P.out.clone()
        saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws)
        return a, P.out.clone()
    alone = [work(P, t) for P, t in zip(Ps, taus)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ps]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(Ps[i], taus[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for pair in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(pair, alone[i]))


def test_offsets_past_32_bits():
    """A second sequence whose codes lie past 2^31 bytes."""
    far = (1 << 32) + 256
    shp = saga.shape(2, 8, 2, 2, 64, saga.SAGA_BF16, 512)
    shp.k_stride_b = shp.v_stride_b = far
    near = Problem(2, 8, 2, 2, 64, saga.SAGA_BF16, 512, [500, 333], 12)
    cache = saga.Q4Cache.__new__(saga.Q4Cache)
    arrays = []
    for src, per in ((near.cache.k_codes, 2), (near.cache.k_scales, 16), (near.cache.v_codes, 2), (near.cache.v_scales, 16)):
        buf = torch.empty(far // per + 2 * 512 * 64 // per, dtype=torch.uint8, device="cuda")
        v = buf.as_strided((2, 2, 512, 64 // per), (far // per, 512 * 64 // per, 64 // per, 1))
        v.copy_(src)
        arrays.append(v)
    cache = saga.Q4Cache(shp, *arrays)
    ws, out = saga.Q4Workspace(shp), torch.zeros(2, 8, 64, device="cuda")
    tau = torch.full((2, 8), 0.5, device="cuda")
    for call in (lambda s, c, o, w: saga.q4_dense_decode(s, c, near.q, near.l, o, w),
                 lambda s, c, o, w: saga.q4_decode_step(s, c, near.q, near.l, tau, o, w)):
        call(near.shp, near.cache, near.out, near.ws)
        call(shp, cache, out, ws)
        assert torch.equal(out, near.out)
    new = torch.randn(2, 1, 2, 64, device="cuda").to(torch.bfloat16)
    got = []
    for s, c, w in ((near.shp, near.cache, near.ws), (shp, cache, ws)):
        l = near.l.clone()
        saga.q4_append_kv(s, c, new, new, 1, l, w)
        K, V = (torch.zeros(2, 2, 40, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        saga.q4_read_kv(s, c, 40, l, K, V, w, start=l - 39)
        got.append((K, V))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][0].any()


def test_against_the_16_bit_calls():
    """Reading the whole cache back and running the 16-bit calls on it: the same
    values in bf16 (exact without head scales), so the same attention within the
    fp32 sums of the two kernels (2e-5 of the largest output) and the same
    thresholds to fp32 rounding of the scores."""
    P = Problem(3, 32, 2, 8, 64, saga.SAGA_BF16, 1300, [1300, 700, 9], 77)
    K = torch.zeros(3, 2, 1300, 64, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros(3, 8, 1300, 64, dtype=torch.bfloat16, device="cuda")
    saga.q4_read_kv(P.shp, P.cache, 1300, P.l, K, V, P.ws)
    ws = saga.Workspace(P.shp, 40)
    out = torch.zeros_like(P.out)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    saga.dense_decode(P.shp, P.q, K, V, P.l, out, ws)
    assert (out - P.out).abs().max() <= 2e-5 * P.out.abs().max()
    tau, tau4 = torch.zeros(3, 32, device="cuda"), torch.zeros(3, 32, device="cuda")
    saga.refresh_threshold(P.shp, P.q, K, P.l, 40, tau, ws)
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, 40, tau4, P.ws)
    live = torch.isfinite(tau)
    assert torch.equal(live, torch.isfinite(tau4))
    assert (tau - tau4)[live].abs().max() <= 2e-5 * tau[live].abs().max()


# ---------------------------------------------------------------------------
# batches and lengths at the ends of the range
# ---------------------------------------------------------------------------
def check_refresh(P, N, rows=None):
    """A refresh with its step: thresholds, masks and outputs against the call's own score rows."""
    tau = torch.full((P.B, P.h_q), float("nan"), device="cuda")
    n = P.shp.max_l_kv
    got = torch.full((P.B, P.h_q, n), 777.0, device="cuda")
    cnt = torch.zeros(P.B, P.h_q, dtype=torch.int32, device="cuda")
    mask = torch.full((P.B, P.h_q, n), 2, dtype=torch.uint8, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out, sel_count=cnt, sel_mask=mask,
                              scores=got)
    assert saga.read_device_error(P.ws) == 0
    r, t = got.cpu().numpy(), tau.cpu().numpy()
    for b in range(P.B):
        for j in range(P.h_q):
            row = r[b, j, :P.lens[b]]
            want = np.float32(orc.nth_largest_f32(row, N)) if row.size else np.float32(-np.inf)
            assert want.view(np.uint32) == t[b, j].view(np.uint32), (b, j)
            if row.size:
                assert np.max(np.abs(row - P.scores(b, j))) <= P.delta(b, j)
    check_step(P, P.out, cnt, mask, tau, rows)
    again = torch.zeros_like(tau)
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, again, P.ws)
    assert torch.equal(tau, again)


@pytest.mark.parametrize("dtype", [saga.SAGA_BF16, saga.SAGA_F32])
@pytest.mark.parametrize("d", [64, 128])
def test_refresh_by_a_bound(d, dtype):
    check_refresh(Problem(5, 8, 2, 4, d, dtype, 8200, [8197, 0, 33, 6500, 512], 51, gscale=True, pad=True), 50)


@pytest.mark.parametrize("N", [1, 3000, 40000])
def test_refresh_longer_than_the_bound_keeps_on_chip(N):
    check_refresh(Problem(1, 3, 1, 1, 64, saga.SAGA_BF16, 150004, [150001], 52), N, rows=[1])


@pytest.mark.parametrize("d", [64, 128])
def test_more_sequences_than_lanes(d):
    lens = np.random.default_rng(3).integers(0, 900, 70)
    lens[::3] = 0
    lens[40:66] = 0
    lens[69] = 900
    P = Problem(70, 4, 1, 2, d, saga.SAGA_BF16, 900, lens, 53)
    saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws)
    P.check_all(P.out)
    check_refresh(P, 30)


def test_rows_of_no_positions():
    P = Problem(3, 8, 2, 4, 64, saga.SAGA_BF16, 4, [0, 0, 0], 54, max_l=0)
    tau = torch.zeros(3, 8, device="cuda")
    saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, 5, tau, P.ws)
    assert torch.all(tau == -np.inf)
    for call in (lambda: saga.q4_dense_decode(P.shp, P.cache, P.q, P.l, P.out, P.ws),
                 lambda: saga.q4_decode_step(P.shp, P.cache, P.q, P.l, tau, P.out, P.ws)):
        P.out.fill_(float("nan"))
        call()
        assert torch.all(P.out == 0) and saga.read_device_error(P.ws) == 0


# ---------------------------------------------------------------------------
# the bounds-checked build: the same results, no check fails
# ---------------------------------------------------------------------------
CHAIN = r"""
import sys
import numpy as np, torch
import sparse_decode_attention_step_b200 as saga
saga.load()
res = {}
for d, hq, hk, hv in ((64, 16, 2, 4), (128, 12, 1, 4)):
    gen = torch.Generator("cuda").manual_seed(d)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()
    shp = saga.shape(3, hq, hk, hv, d, saga.SAGA_BF16, 8200)
    cache, ws = saga.Q4Cache(shp), saga.Q4Workspace(shp)
    l = torch.zeros(3, dtype=torch.int32, device="cuda")
    n = torch.tensor([8190, 0, 301], dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, rand(3, 8190, hk, d), rand(3, 8190, hv, d), 8190, l, ws, n_new=n)
    saga.q4_append_kv(shp, cache, rand(3, 1, hk, d), rand(3, 1, hv, d), 1, l, ws)
    K, V = torch.zeros(3, hk, 300, d, device="cuda").bfloat16(), torch.zeros(3, hv, 300, d, device="cuda").bfloat16()
    saga.q4_read_kv(shp, cache, 300, l, K, V, ws)
    q = rand(3, hq, d)
    out, tau = torch.zeros(3, hq, d, device="cuda"), torch.zeros(3, hq, device="cuda")
    saga.q4_dense_decode(shp, cache, q, l, out, ws)
    dense = out.cpu().numpy().copy()
    saga.q4_refresh_threshold(shp, cache, q, l, 60, tau, ws, out=out)
    fresh = out.cpu().numpy().copy()
    saga.q4_decode_step(shp, cache, rand(3, hq, d), l, tau, out, ws)
    for k, x in (("K", K.float()), ("V", V.float()), ("tau", tau), ("step", out), ("l", l)):
        res[f"d{d}_{k}"] = x.cpu().numpy()
    res[f"d{d}_dense"], res[f"d{d}_fresh"] = dense, fresh
    res[f"d{d}_err"] = np.array([saga.read_device_error(ws)])
np.savez(sys.argv[1], **res)
"""


def test_checked_build_agrees(tmp_path):
    from sparse_decode_attention_step_b200 import build
    if not os.path.exists(build.CHECK_LIB_PATH):
        build.build(check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = []
    for checked in ("0", "1"):
        path = str(tmp_path / f"{checked}.npz")
        env = dict(os.environ, SAGA_CHECKED_BUILD=checked,
                   PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
        r = subprocess.run([sys.executable, "-c", CHAIN, path], env=env, cwd=root, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(np.load(path))
    for k in got[0].files:
        assert np.array_equal(got[0][k], got[1][k]), k
    assert not got[1]["d64_err"].any() and not got[1]["d128_err"].any()


@pytest.mark.parametrize("N", [1, 40, 7000])
def test_nan_and_infinite_queries_in_long_rows(N):
    """The same where the refresh takes its bound from the group maxima."""
    P = Problem(2, 16, 2, 4, 64, saga.SAGA_BF16, 8200, [8197, 6500], 29)
    tau = torch.zeros(2, 16, device="cuda")

    def run():
        saga.q4_refresh_threshold(P.shp, P.cache, P.q, P.l, N, tau, P.ws, out=P.out)
        return tau.clone().cpu(), P.out.clone().cpu()
    clean = run()
    P.q[0, 1, 3] = float("nan")
    P.q[0, 9, :] = float("inf")
    P.q[1, 2, 5] = float("inf")
    P.q[1, 14, :] = float("nan")
    got = run()
    assert saga.read_device_error(P.ws) == 0
    ok = torch.ones(2, 16, dtype=torch.bool)
    for b, j in ((0, 1), (0, 9), (1, 2), (1, 14)):
        ok[b, j] = False
    for x, y in zip(got, clean):
        assert torch.equal(x[ok], y[ok])
