"""The heads' log-probabilities and the draft head's distillation at temperatures far from one, against 64 bits.

Logits are exact sums (values on a grid), maxima from about -30 to 30, so what is off comes from the division by the
temperature and the softmax alone.  Tolerances count those roundings: logits relative to the row's largest carry 5 of
them (the difference, 1 / T, log2 e, their product, the exponent), whatever the size of the largest is."""
import math

import pytest
import torch

import heads_ref as ref
from heads_ref import BF, U
from speculative_decoding_verify_lm_gb300 import wf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TEMPERATURES = [1e30, 100.0, 0.1, 1e-2, 1e-3, 2e-4, 2e-5, 3e-7, 3e-8, 1e-8, 3e-9, 1e-9, 1e-12, 1e-20, 1e-36]
V = 3001


def inputs(P, seed, d=64):
    """x [P, d], W [V, d]: every product a multiple of 2^-11, every sum exact in fp32; rows of all widths, some with
    every logit below zero and some whose largest is there twice."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    W = ref.grid(torch.randn((V, d), device=DEV, generator=g) * 0.5, 2.0 ** -6)
    x = torch.randn((P, d), device=DEV, generator=g) * torch.tensor([0.25, 0.5, 1.0, 1.5], device=DEV).repeat(P)[:P, None]
    x = ref.grid(x, 2.0 ** -5)
    W[:, 0] = 1.0
    x[:, 0] = torch.tensor([0.0, 2.0, -30.0], device=DEV).repeat(P)[:P].to(torch.bfloat16)
    raw = x.double() @ W.double().T
    W[V - 7] = W[raw[1].argmax()]                       # row 1's largest, once more
    return x, W, g


class Row:
    """64-bit softmax over raw / T, and how far fp32 may be off it."""

    def __init__(self, x, W, T):
        self.raw = x.double() @ W.double().T
        assert bool((self.raw.float().double() == self.raw).all())
        self.T = T
        self.top = self.raw.amax(1, keepdim=True)
        self.zz = (self.raw - self.top) / T             # relative to the largest
        e = self.zz.exp()
        s = e.sum(1, keepdim=True)
        self.logs = s.log()
        self.q = e / s
        self.lq = self.zz - self.logs
        self.lse = (self.top / T + self.logs)[:, 0]
        self.mean = -(self.q * self.zz).sum(1)          # of the distance to the largest
        self.square = (self.q * self.zz ** 2).sum(1)
        self.H = self.logs[:, 0] + self.mean
        # sums: a rounding and a rescaling (the exponential's 2 units in the last place, a product) for each group of
        # 32 columns, the partial sums', 160 merged states' the same
        n = W.shape[0] / 32 + 160
        self.es = (6 * n + 20) * U
        # log S: the exponents' 5 roundings, the sum's, the logarithm's
        self.el = 5 * U * self.mean + self.es + 2 * U * self.logs[:, 0]
        self.tol_lse = 2 * U * (self.top[:, 0] / T).abs() + U * self.lse.abs() + self.el
        self.tol_H = self.el + 5 * U * (self.mean + self.square) + 2 * self.es * self.mean + 8 * U * (self.mean + self.H)

    def tol_logp(self, ids):
        return 3 * U * torch.gather(self.zz, 1, ids).abs() + U * torch.gather(self.lq, 1, ids).abs() + self.el[:, None]


def f32(T):
    return float(torch.tensor(T, dtype=torch.float32))


def within(got, want, tol, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), (what, int((~torch.isfinite(got)).sum()))
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("P,k", [(41, 10), (300, 16), (300, 0)])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_logprobs(T, P, k):
    T = f32(T)
    x, W, g = inputs(P, P + k)
    r = Row(x, W, T)
    tok = torch.randint(0, V, (P, 3), device=DEV, generator=g)
    tok[:, 0] = r.raw.argmax(1)
    tok[:, 1] = r.raw.topk(2, 1).indices[:, 1]
    ws = wf.LogprobsWorkspace(P, 64, V, S=3, k=k)
    got = wf.wf_lmhead_logprobs(x, W, ws, tok=tok.int(), k=k, temperature=T, with_entropy=True)
    within(got.lse, r.lse, r.tol_lse, "lse")
    within(got.H, r.H, r.tol_H, "H")
    within(got.logp, torch.gather(r.lq, 1, tok), r.tol_logp(tok), "logp")
    if k:
        best = torch.sort(r.raw, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(got.top_ids, best.int())
        within(got.top_logp, torch.gather(r.lq, 1, best), r.tol_logp(best), "top_logp")


def teacher(r, P, g):
    """Four alternatives a row: its surest id alone, or beside others, falling logits; rows without any."""
    best = r.raw.argmax(1)
    tid = torch.randint(0, V, (P, 4), device=DEV, generator=g)
    tid[:, 0] = best
    tid[::3, 1:] = -1                                    # the surest alone: loss and G are next to nothing
    tid[5::17] = -1
    tl = 10 - torch.empty((P, 4), device=DEV).exponential_(1.0, generator=g).cumsum(1)
    tl[1::3] = 10.0                                      # equal weights at every temperature
    return tid, tl


def loss_of(r, tid, tl, T):
    """The loss in 64 bits, its tolerance, the teacher's ids and probabilities."""
    ids, p, some = ref.teacher(tid.int(), tl, None, T, V)
    lq = torch.gather(r.lq, 1, ids)
    want = torch.where(p > 0, p * (torch.log(torch.where(p > 0, p, 1.0)) - lq), 0.0).sum(1)
    # the teacher's own softmax and sums of up to 4 terms: 250 U of their sizes, as in test_heads_gpu.py
    tol = 250 * U * ((p * lq.abs()).sum(1) + 6) + torch.where(some, r.el, 0.0)
    return want, tol, ids, p, some


@pytest.mark.parametrize("N", [41, 300])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_loss(T, N):
    T = f32(T)
    x, W, g = inputs(N, N)
    r = Row(x, W, T)
    tid, tl = teacher(r, N, g)
    want, tol, *_ = loss_of(r, tid, tl, T)
    loss, lse = wf.wf_draft_distill(x, W, tid.int(), tl, wf.DistillWorkspace(N, 64, V, 4), temperature=T)
    within(lse, r.lse, r.tol_lse, "lse")
    within(loss, want, tol, "loss")
    assert float(loss[5]) == 0


@pytest.mark.parametrize("N", [41, 300])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_kept_logits(T, N):
    """The loss read off kept logits, and the gradients."""
    T = f32(T)
    x, W, g = inputs(N, N)
    r = Row(x, W, T)
    tid, tl = teacher(r, N, g)
    want, tol, ids, p, some = loss_of(r, tid, tl, T)
    # gradients of the size of one whatever the temperature
    gloss = (torch.rand(N, device=DEV, generator=g) + 0.5) * min(T, 1e6)
    ws, z = wf.DistillWorkspace(N, 64, V, 4), wf.distill_logits(N, V)
    loss, lse = wf.wf_draft_distill(x, W, tid.int(), tl, ws, temperature=T, z=z)
    dx, dW = wf.wf_draft_distill_grad(x, W, tid.int(), tl, z, lse, ws, gloss=gloss, temperature=T)
    within(z[:, :V], r.raw / T, 2 * U * (r.raw / T).abs(), "z")
    within(lse, r.lse, r.tol_lse, "lse")
    # kept logits are rounded one by one; the largest's own rounding cancels
    other = torch.gather(r.zz, 1, ids) < 0
    big = (torch.gather(r.raw, 1, ids).abs() + r.top.abs()) / T
    within(loss, want, tol + (p * torch.where(other, U * big, 0.0)).sum(1), "loss")
    assert float(loss[5]) == 0

    gs = torch.where(some, gloss.double() / T, 0.0)[:, None]
    pt = torch.zeros_like(r.q).scatter_add_(1, ids, p)
    G = gs * (r.q - pt)
    # q = e^(z - lse): kept logits' roundings but the largest's; lse's own, half a step of it and no more than log S, by
    # which it lies beside a number of fp32, the largest kept logit; their difference's
    ez = torch.where(r.zz < 0, U * (r.raw.abs() + r.top.abs()) / T, 0.0) + torch.minimum(r.logs, U * r.lse[:, None].abs())
    ez = ez + 3 * U * r.zz.abs() + r.el[:, None] + 4 * U * r.lq.abs() + 4 * U
    eq = (r.lq + ez).clamp(max=30).exp() - r.q
    eG = (BF if N > 128 else BF * BF) * G.abs() + gs * (eq + pt * 250 * U) * (1 + 4 * U)
    # below 2^-126 there are no normal numbers: the exponential gives 0 there (a q of up to 2^-126, times gs), and a part
    # of G that small, or the second part of a larger one, may count as 0 (2^-126 each)
    eG = eG + (gs + 2) * 2.0 ** -126
    Wd, X = W.double(), x.double()
    gx, gW = G @ Wd, G.T @ X
    tx = (1 + BF) * (eG @ Wd.abs() + 4 * V * U * (G.abs() @ Wd.abs())) + BF * gx.abs() + 1e-38
    tW = (1 + BF) * (eG.T @ X.abs() + 4 * N * U * (G.abs().T @ X.abs())) + BF * gW.abs() + 1e-38
    within(dx, gx, tx, "dx")
    within(dW, gW, tW, "dWd")
