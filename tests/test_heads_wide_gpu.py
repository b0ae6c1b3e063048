"""Wide states: the splits of dx that only they take, and log-probabilities of more than one launch's rows whose pairs
share what their best have reached."""
import pytest
import torch

import heads_ref as ref
from speculative_decoding_verify_lm_gb300 import wf
from test_heads_gpu import DEV, check_logprobs, check_loss, gen, step, teacher_of, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [20, 100, 300])
@pytest.mark.parametrize("d,Vd", [(4096, 1503), (4096, 9000), (10000, 3001), (16384, 700), (16384, 5000)])
def test_distill(N, d, Vd):
    """d 10,000 and 16,384: more column tiles than half the pairs, so that 20 rows are not split."""
    g = gen(N + d)
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.01)
    tid, tl, t2d = teacher_of(N, Vd, 6, 2 * Vd, g)
    gloss = torch.rand(N, device=DEV, generator=g) / N
    loss, lse, z, dx, dW = step(x, Wd, tid, tl, t2d, 1.0, gloss)
    want = ref.distill(x, Wd, tid, tl, t2d, 1.0)
    within(z[:, :Vd], want["z"], 3 * ref.U * want["z"].abs() + 1e-38, "z")
    check_loss(loss, lse, want, 1.0, Vd)
    gx, gW, tx, tW = ref.grads(x, Wd, want, gloss, 1.0)
    within(dx, gx, tx, "dx")
    within(dW, gW, tW, "dWd")
    ws = wf.DistillWorkspace(N, d, Vd, 6)
    only, _ = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, gloss=gloss, t2d=t2d, need_dWd=False)
    within(only, gx, tx, "dx alone")
    _, only = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, gloss=gloss, t2d=t2d, need_dx=False)
    assert torch.equal(only, dW)


@pytest.mark.parametrize("k", [10, 16])
def test_logprobs_of_several_launches_rows(k):
    """3,000 rows of 16,384 go in launches of 1,536 and 1,464, each of six row tiles and about 80 weight tiles; the second
    has other rows where the first put its maxima down, lower ones."""
    g = gen(40 + k)
    P, d, V = 3000, 16384, 20000
    W, h = ref.head(V, d, g, std=0.005), ref.states(P, d, g)
    h[1536:] = ref.grid(h[1536:].float() / 4, 2.0 ** -5)
    tok = torch.randint(0, V, (P, 2), device=DEV, generator=g).int()
    ws = wf.LogprobsWorkspace(P, d, V, S=2, k=k)
    r = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=k, with_entropy=True)
    want, tol = ref.logprobs(h, W, 1.0, tok, k)
    check_logprobs(r, want, tol, k)
    again = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=k, with_entropy=True)
    assert all(torch.equal(a, b) for a, b in zip(again, r))
