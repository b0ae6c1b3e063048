"""A teacher's row that names one draft id in several places: the loss takes the places apart, the gradient adds them."""
import math

import pytest
import torch

import heads_ref as ref
from heads_ref import U
from speculative_decoding_verify_lm_gb300 import wf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("N", [5, 200])
def test_two_places_of_a_sure_id(N):
    """Two equal places of an id that the student is sure of: 2 (1/2 log 1/2) = -log 2, and no gradient."""
    W = torch.zeros((700, 64), dtype=torch.bfloat16, device=DEV)
    W[77, 0] = 1.0
    x = torch.zeros((N, 64), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 200.0                                      # q of id 77: 1 - 700 e^-200
    tid = torch.tensor([[77, -1, 77]], dtype=torch.int32, device=DEV).repeat(N, 1)
    tl = torch.full((N, 3), 3.0, device=DEV)
    ws, z = wf.DistillWorkspace(N, 64, 700, 3), wf.distill_logits(N, 700)
    for kept in (None, z):
        loss, lse = wf.wf_draft_distill(x, W, tid, tl, ws, z=kept)
        # log 2 and its sum: a few roundings of numbers below one
        assert bool(((loss.double() + math.log(2)).abs() <= 8 * U).all())
        assert bool(((lse.double() - 200).abs() <= 200 * U).all())
    dx, dW = wf.wf_draft_distill_grad(x, W, tid, tl, z, lse, ws)
    # G is q - 2 (1/2): 0, or the roundings of q
    assert float(dx.float().abs().max()) <= 8 * U and float(dW.float().abs().max()) <= 8 * U * 200 * N


@pytest.mark.parametrize("N", [40, 200])
def test_ids_that_the_map_brings_together(N):
    """Target ids 2 i and 2 i + 1 are draft id i.  Loss: the sum over the places.  Gradients: those of one place with both
    probabilities."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N)
    d, Vd, k = 128, 900, 6
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.05)
    t2d = (torch.arange(2 * Vd, device=DEV) // 2).int()
    ids = torch.rand((N, Vd), device=DEV, generator=g).argsort(1)[:, :k // 2]
    tid = torch.stack((2 * ids, 2 * ids + 1), 2).reshape(N, k).int()
    tl = torch.randn((N, k), device=DEV, generator=g)
    ws, z = wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)
    loss, lse = wf.wf_draft_distill(x, Wd, tid, tl, ws, t2d=t2d, z=z)
    dx, dW = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, t2d=t2d)
    logits = ref.logits(x, Wd, 1.0)
    lq = logits - torch.logsumexp(logits, 1, keepdim=True)
    p = torch.softmax(tl.double(), 1)
    places = torch.gather(lq, 1, tid.long() // 2)
    apart = (p * (p.log() - places)).sum(1)
    both = p.reshape(N, k // 2, 2).sum(2)
    kl = (both * (both.log() - torch.gather(lq, 1, ids))).sum(1)
    tol = 2 * (5 * U * logits.abs().amax(1)) + ref.sum_error(Vd) + 250 * U * ((p * places.abs()).sum(1) + 6)
    assert bool(((loss.double() - apart).abs() <= tol).all())
    assert float((kl - apart > tol).double().mean()) > 0.9   # the divergence is more, by what tells the places apart
    want = ref.distill(x, Wd, ids.int(), both.log().float(), None, 1.0)
    gx, gW, tx, tW = ref.grads(x, Wd, want, None, 1.0)
    assert bool(((dx.double() - gx).abs() <= tx).all()) and bool(((dW.double() - gW).abs() <= tW).all())
