"""A score pass that gave up a bounded wait leaves the workspace's abort word (the
one behind the error word) set. The call that it belongs to poisons its results and
clears the word; the next call on the workspace is whole. The word is set by
hand here: to the rest of the call that is what a give-up leaves. The last test runs the
waits out, in a build whose waits are short."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_decode_attention_step_b200 as saga

pytestmark = pytest.mark.gpu

B, H_Q, H_K, H_V, D, N = 3, 16, 2, 4, 64, 40


@pytest.fixture(scope="module", autouse=True)
def _built(gpu_lib):
    return gpu_lib


class Sixteen:
    """The calls over a 16-bit cache, and (Four) over a 4-bit one."""

    def __init__(self, cap):
        gen = torch.Generator("cuda").manual_seed(cap)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()
        self.shp = saga.shape(B, H_Q, H_K, H_V, D, saga.SAGA_BF16, cap)
        self.K, self.V, self.q = rand(B, H_K, cap, D), rand(B, H_V, cap, D), rand(B, H_Q, D)
        self.l = torch.tensor([cap - 3, N - 1, 700], dtype=torch.int32, device="cuda")
        self.tau = torch.zeros(B, H_Q, device="cuda")
        self.out = torch.zeros(B, H_Q, D, device="cuda")
        self.cnt = torch.zeros(B, H_Q, dtype=torch.int32, device="cuda")
        self.make()
        self.word = self.ws.buf[4:8].view(torch.int32)

    def make(self):
        self.ws = saga.Workspace(self.shp, N)

    def refresh(self, out):
        saga.refresh_threshold(self.shp, self.q, self.K, self.l, N, self.tau, self.ws, V=self.V if out else None,
                               out=self.out if out else None, sel_count=self.cnt if out else None)

    def step(self):
        saga.decode_step(self.shp, self.q, self.K, self.V, self.l, self.tau, self.out, self.ws, sel_count=self.cnt)


class Four(Sixteen):
    def make(self):
        self.cache, self.ws = saga.Q4Cache(self.shp), saga.Q4Workspace(self.shp)
        l, cap = torch.zeros(B, dtype=torch.int32, device="cuda"), self.shp.cap
        saga.q4_append_kv(self.shp, self.cache, self.K.transpose(1, 2).contiguous(),
                          self.V.transpose(1, 2).contiguous(), cap, l, self.ws)

    def refresh(self, out):
        saga.q4_refresh_threshold(self.shp, self.cache, self.q, self.l, N, self.tau, self.ws,
                                  out=self.out if out else None, sel_count=self.cnt if out else None)

    def step(self):
        saga.q4_decode_step(self.shp, self.cache, self.q, self.l, self.tau, self.out, self.ws, sel_count=self.cnt)


def check(P):
    P.refresh(False)
    P.step()
    tau, out, cnt = P.tau.clone(), P.out.clone(), P.cnt.clone()
    assert torch.isfinite(out).all() and torch.all(tau[1] == -torch.inf) and torch.isfinite(tau[::2]).all()

    # thresholds alone: none from the scores of a pass that gave up (a short row's is
    # -inf whatever they are), and the word is cleared for the next call
    P.word.fill_(1)
    P.refresh(False)
    assert torch.isnan(P.tau[::2]).all() and torch.all(P.tau[1] == -torch.inf)
    assert P.word.item() == 0
    P.tau.copy_(tau)
    P.step()
    assert torch.equal(P.out, out) and torch.equal(P.cnt, cnt)
    P.refresh(False)
    assert torch.equal(P.tau, tau)

    # the refresh with its step, and the step
    for call in (lambda: P.refresh(True), P.step):
        P.word.fill_(1)
        call()
        assert torch.isnan(P.out).all() and torch.all(P.cnt == -1) and P.word.item() == 0
        P.refresh(True)
        assert torch.equal(P.tau, tau) and torch.equal(P.cnt, cnt)
        P.step()
        assert torch.equal(P.out, out)


@pytest.mark.parametrize("cap", [1300, 8200])              # without and with the bound
def test_q4_refresh(cap):
    check(Four(cap))


def test_refresh():
    check(Sixteen(1300))


def test_score_rows_alone_leave_the_word():
    """The rows that saga_debug_scores writes are no part of a step: it neither reads nor clears the word."""
    P = Sixteen(1300)
    P.word.fill_(1)
    saga.debug_scores(P.shp, P.q, P.K, P.l, torch.zeros(B, H_Q, 1300, device="cuda"), P.ws)
    assert P.word.item() == 1
    P.step()
    assert torch.isnan(P.out).all() and P.word.item() == 0


# The waits themselves: in the short-wait build the 4-bit kernels give up wherever a copy
# has not landed yet, with the copies they issued in flight.
CHAIN = r"""
import sys
import numpy as np, torch
import sparse_decode_attention_step_b200 as saga
saga.load()
res = {}
# rows long enough for several chunks a CTA, and caches pushed out of L2: a first chunk, or
# one from L2, often lands behind the query's loads
B, away = 12, torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
for d, heads, cap, dt in ((64, (16, 2, 4), 32768, 1), (128, (12, 1, 4), 32768, 1), (64, (8, 8, 8), 6000, 0),
                          (128, (16, 1, 1), 32768, 0)):
    gen = torch.Generator("cuda").manual_seed(d)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16 if dt else torch.float32)
    shp = saga.shape(B, *heads, d, saga.SAGA_BF16 if dt else saga.SAGA_F32, cap)
    cache, ws = saga.Q4Cache(shp), saga.Q4Workspace(shp)
    l = torch.zeros(B, dtype=torch.int32, device="cuda")
    n = torch.tensor([cap - 2, 0, 301] + [cap - 3] * (B - 3), dtype=torch.int32, device="cuda")
    saga.q4_append_kv(shp, cache, rand(B, cap, heads[1], d), rand(B, cap, heads[2], d), cap, l, ws, n_new=n)
    q, word = rand(B, heads[0], d), ws.buf[4:8].view(torch.int32)
    out, tau = torch.zeros(B, heads[0], d, device="cuda"), torch.zeros(B, heads[0], device="cuda")
    cnt = torch.zeros(B, heads[0], dtype=torch.int32, device="cuda")
    for name, call in (("dense", lambda: saga.q4_dense_decode(shp, cache, q, l, out, ws)),
                       ("tau", lambda: saga.q4_refresh_threshold(shp, cache, q, l, 60, tau, ws)),
                       ("fresh", lambda: saga.q4_refresh_threshold(shp, cache, q, l, 60, tau, ws, out=out,
                                                                   sel_count=cnt)),
                       ("step", lambda: saga.q4_decode_step(shp, cache, q, l, torch.zeros_like(tau), out, ws,
                                                            sel_count=cnt))):
        away.fill_(1), out.zero_(), tau.zero_(), cnt.zero_()
        call()
        err = saga.read_device_error(ws)
        for k, x in (("out", out), ("tau", tau), ("cnt", cnt)):
            res[f"{d}{heads} {name} {k}"] = x.cpu().numpy()
        res[f"{d}{heads} {name} err"] = np.array([err, word.item()])
np.savez(sys.argv[1], **res)
"""


def test_q4_waits_that_run_out(tmp_path):
    from sparse_decode_attention_step_b200 import build
    if not os.path.exists(build.SHORT_LIB_PATH):
        build.build(short_waits=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = []
    for short in ("0", "1"):
        path = str(tmp_path / f"{short}.npz")
        env = dict(os.environ, SAGA_CHECKED_BUILD="0", SAGA_SHORT_WAITS_BUILD=short,
                   PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""))
        r = subprocess.run([sys.executable, "-c", CHAIN, path], env=env, cwd=root, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(np.load(path))
    plain, short = got
    gave_up = set()
    for k in [k[:-4] for k in plain.files if k.endswith(" err")]:
        kind = k.split()[-1]
        assert plain[k + " err"].tolist() == [0, 0]
        err, word = short[k + " err"].tolist()
        assert err in (0, 4) and word == 0, k              # SAGA_DEVERR_TIMEOUT; the abort word is cleared
        a, b = ({x: r[f"{k} {x}"] for x in ("out", "tau", "cnt")} for r in (plain, short))
        if err == 0:
            assert all(np.array_equal(a[x], b[x]) for x in a), k
            continue
        gave_up.add(kind)
        if kind == "dense":
            # rows whose CTAs all had their copies in time are whole, the others NaN throughout
            nan = np.isnan(b["out"]).all(-1)
            assert np.array_equal(np.isnan(b["out"]).any(-1), nan) and nan.any(), k
            assert np.array_equal(a["out"][~nan], b["out"][~nan]) and not b["out"][1].any(), k
        if kind in ("tau", "fresh"):
            assert np.isnan(np.delete(b["tau"], 1, 0)).all() and np.all(b["tau"][1] == -np.inf), k
        if kind in ("fresh", "step"):
            assert np.isnan(b["out"]).all() and np.all(b["cnt"] == -1), k
    assert gave_up == {"dense", "tau", "fresh", "step"}
