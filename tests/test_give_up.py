"""A score pass that gave up a bounded wait leaves the workspace's abort word (the
one behind the error word) set. The call that it belongs to poisons its results and
clears the word; the next call on the workspace is whole. The word is set by
hand here: to the rest of the call that is what a give-up leaves."""
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
