"""Best alternatives of rows whose k-th best logit is exactly zero (a padded batch's rows of zeros, rows for which few
ids have a logit above zero), and of rows that many pairs of CTAs see tile after tile, whose best bound each other."""
import pytest
import torch

import heads_ref as ref
from speculative_decoding_verify_lm_gb300 import wf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(h, W, k):
    P, V = h.shape[0], W.shape[0]
    tok = torch.arange(P, device=DEV).int() % V
    r = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(P, h.shape[1], V, S=1, k=k), tok=tok, k=k, with_entropy=True)
    want, tol = ref.logprobs(h, W, 1.0, tok, k)
    assert torch.equal(r.top_ids, want["top_ids"])
    assert bool(((r.top_logp.double() - want["top_logp"]).abs() <= tol["logp"][:, None]).all())
    assert bool(((r.logp.double() - want["logp"]).abs() <= tol["logp"]).all())


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("P,V,k", [(5, 1, 1), (5, 300, 4), (60, 41000, 10), (300, 700, 16), (700, 50021, 10),
                                   (2100, 9001, 3)])
def test_rows_of_zeros(P, V, k, sign):
    """Every logit is zero, of either sign: the k lowest ids."""
    g = torch.Generator(device=DEV)
    g.manual_seed(P + V)
    W, h = ref.head(V, 64, g, std=0.1), ref.states(P, 64, g)
    h[P // 3:] = sign * 0.0
    check(h, W, k)


@pytest.mark.parametrize("P,V,k", [(40, 41000, 10), (300, 50021, 16), (1030, 9001, 4)])
def test_few_ids_above_zero(P, V, k):
    """A few ids' logits are not zero, and about half of those lie below it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(P)
    W, h = torch.zeros((V, 64), dtype=torch.bfloat16, device=DEV), ref.states(P, 64, g)
    some = torch.arange(V // 2, V, 5000, device=DEV)
    W[some] = ref.head(some.numel(), 64, g, std=0.1)
    check(h, W, k)


@pytest.mark.parametrize("P,V,k", [(700, 50021, 10), (1500, 30011, 16), (400, 60001, 1)])
def test_many_tiles_of_the_same_rows(P, V, k):
    """Eager, captured and replayed on new inputs, with logits that rise with the id, fall with it or lie anyhow."""
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    W, h = ref.head(V, 64, g, std=0.05), ref.states(P, 64, g)
    W[:, 0] = (torch.arange(V, device=DEV) // 512 * 2.0 ** -5).to(torch.bfloat16)   # 2 to 8 bits, exact
    h[:, 0] = torch.tensor([0.0, 2.0, -2.0], device=DEV).repeat(P)[:P].to(torch.bfloat16)
    ws = wf.LogprobsWorkspace(P, 64, V, k=k)
    buf = h.clone()
    wf.wf_lmhead_logprobs(buf, W, ws, k=k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wf.wf_lmhead_logprobs(buf, W, ws, k=k, with_entropy=True)
    for shift in (0, 1, 2):
        new = h.roll(shift, 0).contiguous()
        eager = wf.wf_lmhead_logprobs(new, W, ws, k=k, with_entropy=True)
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ref.logprobs(new, W, 1.0, None, k)
        for r in (eager, out):
            assert torch.equal(r.top_ids, want["top_ids"])
            assert bool(((r.top_logp.double() - want["top_logp"]).abs() <= tol["logp"][:, None]).all())
        assert torch.equal(eager.lse, out.lse) and torch.equal(eager.H, out.H)
