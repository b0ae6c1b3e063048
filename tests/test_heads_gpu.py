"""The heads' log-probabilities and the draft head's distillation on the GPU against plain 64-bit references."""
import math

import pytest
import torch

import heads_ref as ref
from speculative_decoding_verify_lm_gb300 import wf
from test_canary_gpu import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BAD_DATA = 5


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def within(got, want, tol, what):
    got = got.double()
    bad = (got - want).abs() > tol
    assert not bool(bad.any()) and bool(torch.isfinite(got).all()), (
        what, int(bad.sum()), float(((got - want).abs() / tol).max()))


def rows(tol, like):
    return tol.reshape(-1, *([1] * (like.dim() - 1)))


def check_logprobs(r, want, tol, k):
    within(r.lse, want["lse"], tol["lse"], "lse")
    within(r.H, want["H"], tol["H"], "H")
    if want["logp"] is not None:
        within(r.logp, want["logp"], rows(tol["logp"], r.logp), "logp")
    if k:
        assert torch.equal(r.top_ids, want["top_ids"])
        within(r.top_logp, want["top_logp"], rows(tol["logp"], r.top_logp), "top_logp")


# ------------------------------------------------------------------ log-probabilities
@pytest.mark.parametrize("P,d,V,S,k,T", [
    (1, 8, 1, 1, 1, 1.0), (1, 64, 5, 3, 5, 0.5), (3, 256, 1000, 1, 0, 1.0), (17, 256, 8192, 0, 3, 2.0),
    (61, 256, 4999, 10, 10, 1.0), (128, 72, 33, 64, 16, 1.0), (127, 1000, 20011, 2, 11, 0.7),
    (129, 64, 257, 1, 4, 1.0), (130, 256, 4999, 5, 16, 1.0), (255, 512, 2048, 1, 1, 1.3), (256, 256, 30000, 1, 10, 1.0),
    (257, 256, 255, 16, 10, 1.0), (515, 128, 31000, 3, 9, 1.0), (2100, 136, 5003, 1, 16, 1.0),
    (2304, 64, 700, 0, 10, 1.0), (16500, 64, 300, 1, 2, 1.0), (40, 2560, 39000, 1, 16, 1.0),
])
def test_logprobs(P, d, V, S, k, T):
    g = gen(P + V)
    W, h = ref.head(V, d, g, std=0.5 / math.sqrt(d) if d < 256 else 0.02), ref.states(P, d, g)
    tok = None
    if S:
        tok = torch.randint(-1, V, (P, S), device=DEV, generator=g).int()
        tok = tok[:, 0].contiguous() if S == 1 and P % 2 else tok
    ws = wf.LogprobsWorkspace(P, d, V, S=S, k=k)
    r = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=k, temperature=T, with_entropy=True)
    want, tol = ref.logprobs(h, W, T, tok, k)
    check_logprobs(r, want, tol, k)
    assert ws.device_error() == (0, 0)


@pytest.mark.parametrize("P,V", [(9, 3001), (300, 3001)])
def test_logprobs_of_any_bf16_values(P, V):
    """Off the grid: logits to fp32's sums; ranks where the gaps are wider than that."""
    g = gen(5)
    W, h = ref.head(V, 2560, g, on_grid=False), ref.states(P, 2560, g, on_grid=False)
    tok = torch.randint(0, V, (P, 2), device=DEV, generator=g).int()
    r = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(P, 2560, V, S=2, k=10), tok=tok, k=10, with_entropy=True)
    want, tol = ref.logprobs(h, W, 1.0, tok, 10, on_grid=False)
    within(r.top_logp, want["top_logp"], rows(tol["logp"], r.top_logp), "top_logp")
    clear = torch.ones(P, 10, dtype=torch.bool, device=DEV)
    gap = want["top_logp"][:, :-1] - want["top_logp"][:, 1:]
    clear[:, 1:] &= gap > 2 * rows(tol["logp"], gap)
    clear[:, :-1] &= gap > 2 * rows(tol["logp"], gap)
    clear[:, 9] = False
    assert bool(clear.any()) and torch.equal(r.top_ids[clear], want["top_ids"][clear])
    want["top_ids"] = r.top_ids
    check_logprobs(r, want, tol, 10)


@pytest.mark.parametrize("P", [5, 140])
def test_equal_logits_rank_by_id(P):
    """Rows of W that are equal, in one tile, in neighbouring ones and far apart."""
    g = gen(11)
    base = ref.head(37, 128, g, std=0.05)
    W = base[torch.randint(0, 37, (9001,), device=DEV, generator=g)].contiguous()
    h = ref.states(P, 128, g)
    r = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(P, 128, 9001, k=16), k=16, with_entropy=True)
    want, tol = ref.logprobs(h, W, 1.0, None, 16)
    check_logprobs(r, want, tol, 16)


@pytest.mark.parametrize("P", [20, 333])
def test_a_given_token_has_an_alternatives_bits(P):
    g = gen(12)
    W, h = ref.head(5000, 256, g, on_grid=False), ref.states(P, 256, g, on_grid=False)
    ws = wf.LogprobsWorkspace(P, 256, 5000, S=16, k=16)
    best = wf.wf_lmhead_logprobs(h, W, ws, k=16, with_entropy=True)
    perm = torch.randperm(16, device=DEV, generator=g)
    tok = best.top_ids[:, perm].contiguous()
    r = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=16, with_entropy=True)
    assert torch.equal(r.logp, best.top_logp[:, perm]) and torch.equal(r.lse, best.lse) and torch.equal(r.H, best.H)
    # the same token several times, and one column only
    twice = tok[:, [3, 3, 0, 3]].contiguous()
    r2 = wf.wf_lmhead_logprobs(h, W, ws, tok=twice, k=0)
    assert torch.equal(r2.logp, r.logp[:, [3, 3, 0, 3]]) and r2.H is None and r2.top_ids is None
    r1 = wf.wf_lmhead_logprobs(h, W, ws, tok=tok[:, 5].contiguous())
    assert r1.logp.shape == (P,) and torch.equal(r1.logp, r.logp[:, 5])


@pytest.mark.parametrize("P,S", [(9, 1), (9, 4), (200, 1), (200, 4)])
def test_tokens_out_of_range(P, S):
    g = gen(13)
    V = 2000
    W, h = ref.head(V, 64, g, std=0.1), ref.states(P, 64, g)
    tok = torch.randint(0, V, (P, S), device=DEV, generator=g).int()
    tok[3, 0], tok[4, S - 1], tok[5, 0], tok[6, 0] = V, -2, -1, 2 ** 31 - 1
    ws = wf.LogprobsWorkspace(P, 64, V, S=S)
    r = wf.wf_lmhead_logprobs(h, W, ws, tok=tok)
    want, tol = ref.logprobs(h, W, 1.0, tok.clamp(min=-1, max=V - 1), 0)
    bad = (tok < -1) | (tok >= V)
    assert bool(torch.isnan(r.logp[bad]).all()) and bool((r.logp[tok == -1] == 0).all())
    within(r.logp[~bad], want["logp"][~bad], rows(tol["logp"], r.logp).expand_as(r.logp)[~bad], "logp")
    code, info = ws.device_error()
    assert code == BAD_DATA and info in (3, 4, 6)
    assert ws.device_error() == (0, 0)


@pytest.mark.parametrize("P", [40, 300])
def test_rows_that_are_not_finite_stay_with_themselves(P):
    g = gen(14)
    W, h = ref.head(3000, 128, g, std=0.05), ref.states(P, 128, g)
    tok = torch.randint(0, 3000, (P,), device=DEV, generator=g).int()
    ws = wf.LogprobsWorkspace(P, 128, 3000, S=1, k=4)
    clean = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=4, with_entropy=True)
    sick = h.clone()
    sick[2], sick[P - 1, 7], sick[33, 0] = math.nan, math.nan, math.inf
    r = wf.wf_lmhead_logprobs(sick, W, ws, tok=tok, k=4, with_entropy=True)
    ill = torch.zeros(P, dtype=torch.bool, device=DEV)
    ill[[2, 33, P - 1]] = True
    for a, b in zip(r, clean):
        assert torch.equal(a[~ill], b[~ill])
    assert bool(torch.isnan(r.lse[ill]).all()) and bool(torch.isnan(r.H[ill]).all())
    assert bool((r.top_ids[[2, P - 1]] == -1).all()) and bool(torch.isnan(r.top_logp[2]).all())


def test_logprobs_of_a_head_past_32_bit_offsets():
    """151,936 x 16,384 weights: 2.5e9 elements; the last ids lie past 2^31."""
    g = gen(15)
    V, d, P = 151936, 16384, 3
    W = torch.zeros((V, d), dtype=torch.bfloat16, device=DEV)
    for v in range(0, V, 8192):
        W[v:v + 8192] = ref.head(min(8192, V - v), d, g, std=0.005)
    h = ref.states(P, d, g)
    tok = torch.tensor([V - 1, 0, 140000], dtype=torch.int32, device=DEV)
    h[0] += (W[V - 1].float() * 300).to(torch.bfloat16)
    h = ref.grid(h.float(), 2.0 ** -5)
    r = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(P, d, V, S=1, k=3), tok=tok, k=3, with_entropy=True)
    raw = torch.cat([h.double() @ W[v:v + 8192].double().T for v in range(0, V, 8192)], 1)
    assert torch.equal(r.top_ids, torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :3].int())
    assert int(r.top_ids[0, 0]) == V - 1
    lse = torch.logsumexp(raw, 1)
    tol = ref.sum_error(V) + 20 * ref.U * raw.abs().amax(1)
    within(r.lse, lse, tol, "lse")
    within(r.logp, raw[torch.arange(P, device=DEV), tok.long()] - lse, tol, "logp")


def test_logprobs_write_their_outputs_only():
    for P in (37, 259):
        g = gen(16)
        W, h = ref.head(4999, 128, g, std=0.05), ref.states(P, 128, g)
        tok = torch.randint(0, 4999, (P, 3), device=DEV, generator=g).int()
        out = dict(logp=Guarded((P, 3), torch.float32), lse=Guarded((P,), torch.float32), H=Guarded((P,), torch.float32),
                   top_ids=Guarded((P, 7), torch.int32), top_logp=Guarded((P, 7), torch.float32))
        r = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(P, 128, 4999, S=3, k=7), tok=tok, k=7,
                                  **{n: o.t for n, o in out.items()})
        want, tol = ref.logprobs(h, W, 1.0, tok, 7)
        check_logprobs(r, want, tol, 7)
        assert all(o.intact() for o in out.values())


def test_logprobs_do_not_read_what_a_workspace_held():
    """Any bytes behind the control block, calls of other shapes before, and the same bits again."""
    g = gen(17)
    W, h = ref.head(6000, 128, g, std=0.05), ref.states(700, 128, g)
    tok = torch.randint(-1, 6000, (700, 4), device=DEV, generator=g).int()
    ws = wf.LogprobsWorkspace(700, 128, 6000, S=4, k=16)
    first = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=16, with_entropy=True)
    for fill in (0xFF, 0x7F, 0x00):
        ws.buf[256:] = fill
        wf.wf_lmhead_logprobs(h[:60].contiguous(), W[:900].contiguous(), ws, tok=tok[:60].clamp(max=899).contiguous(),
                              k=3, with_entropy=True)
        again = wf.wf_lmhead_logprobs(h, W, ws, tok=tok, k=16, with_entropy=True)
        assert all(torch.equal(a, b) for a, b in zip(again, first))


# ------------------------------------------------------------------ distillation
def teacher_of(N, Vd, k, V, g, empty=0.1):
    """Ids (target ids, some without a draft id, if V) and falling logits; some places and rows without a teacher."""
    ids = torch.stack([torch.randperm(max(Vd, k), device=DEV, generator=g)[:k] % Vd for _ in range(min(N, 50))])
    ids = ids[torch.arange(N, device=DEV) % ids.shape[0]]
    ids = (ids + torch.arange(N, device=DEV)[:, None]) % Vd
    logit = 10 - torch.empty((N, k), device=DEV).exponential_(1.0, generator=g).cumsum(1)
    t2d = None
    if V:
        d2t = torch.randperm(V, device=DEV, generator=g)[:Vd]
        t2d = torch.full((V,), -1, dtype=torch.int32, device=DEV)
        t2d[d2t] = torch.arange(Vd, dtype=torch.int32, device=DEV)
        ids = torch.where(torch.rand((N, k), device=DEV, generator=g) < 0.2,
                          torch.randint(0, V, (N, k), device=DEV, generator=g), d2t[ids])
    ids = torch.where(torch.rand((N, k), device=DEV, generator=g) < 0.1, -1, ids)
    ids = torch.where(torch.rand((N, 1), device=DEV, generator=g) < empty, -1, ids)
    return ids.int().contiguous(), logit, t2d


def check_loss(loss, lse, want, T, Vd):
    ez = 5 * ref.U * want["z"].abs().amax(1)
    es = ref.sum_error(Vd)
    within(lse, want["lse"], 2 * ez + es + 4 * ref.U * want["lse"].abs(), "lse")
    # sum p log p and sum p log q: the terms' roundings, p's own (80 U), the sums' of up to 64 terms
    size = (want["p"] * (want["lse"][:, None] - torch.gather(want["z"], 1, want["ids"])).abs()).sum(1) + 6
    within(loss, want["loss"], 2 * ez + es + 250 * ref.U * size, "loss")


def step(x, Wd, tid, tl, t2d, T, gloss, **kw):
    N, d = x.shape
    Vd = Wd.shape[0]
    ws = wf.DistillWorkspace(N, d, Vd, tid.shape[1])
    z = wf.distill_logits(N, Vd)
    loss, lse = wf.wf_draft_distill(x, Wd, tid, tl, ws, t2d=t2d, temperature=T, z=z)
    dx, dW = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, gloss=gloss, t2d=t2d, temperature=T, **kw)
    assert ws.device_error() == (0, 0)
    return loss, lse, z, dx, dW


@pytest.mark.parametrize("N,d,Vd,k,V,T", [
    (1, 8, 1, 1, 0, 1.0), (1, 64, 5, 3, 0, 1.0), (3, 72, 100, 4, 300, 2.0), (17, 256, 1003, 10, 0, 0.5),
    (64, 320, 8000, 10, 20000, 1.0), (64, 1024, 32000, 10, 0, 1.0), (127, 256, 2049, 64, 5000, 1.0),
    (128, 128, 600, 1, 0, 1.0), (129, 264, 777, 5, 0, 1.0), (256, 512, 512, 16, 700, 1.3), (300, 256, 10007, 7, 0, 1.0),
    (777, 136, 4096, 16, 0, 1.0), (2100, 64, 3001, 10, 9000, 1.0), (600, 2560, 1500, 33, 0, 1.0),
    (40, 2560, 39000, 64, 0, 1.0),
])
def test_distill(N, d, Vd, k, V, T):
    g = gen(N + Vd)
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.5 / math.sqrt(d) if d < 256 else 0.02)
    tid, tl, t2d = teacher_of(N, Vd, k, V, g)
    gloss = None if N % 2 else torch.randn(N, device=DEV, generator=g) / N
    loss, lse, z, dx, dW = step(x, Wd, tid, tl, t2d, T, gloss)
    want = ref.distill(x, Wd, tid, tl, t2d, T)
    within(z[:, :Vd], want["z"], 3 * ref.U * want["z"].abs() + 1e-38, "z")
    check_loss(loss, lse, want, T, Vd)
    gx, gW, tx, tW = ref.grads(x, Wd, want, gloss, T)
    within(dx, gx, tx, "dx")
    within(dW, gW, tW, "dWd")
    # the loss alone, and either gradient alone
    ws = wf.DistillWorkspace(N, d, Vd, k)
    l2, s2 = wf.wf_draft_distill(x, Wd, tid, tl, ws, t2d=t2d, temperature=T)
    check_loss(l2, s2, want, T, Vd)
    only, none = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, gloss=gloss, t2d=t2d, temperature=T,
                                          need_dWd=False)
    assert none is None
    within(only, gx, tx, "dx alone")
    none, only = wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws, gloss=gloss, t2d=t2d, temperature=T,
                                          need_dx=False)
    assert none is None and torch.equal(only, dW)


@pytest.mark.parametrize("N", [30, 200])
def test_gradients_against_differences(N):
    """The 64-bit loss's central differences along random directions, against the kernels' gradients."""
    g = gen(21)
    d, Vd, T = 96, 700, 1.5
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.08)
    tid, tl, t2d = teacher_of(N, Vd, 6, 0, g)
    gloss = torch.rand(N, device=DEV, generator=g)
    _, _, _, dx, dW = step(x, Wd, tid, tl, None, T, gloss)
    want = ref.distill(x, Wd, tid, tl, None, T)
    _, _, tx, tW = ref.grads(x, Wd, want, gloss, T)
    f = lambda a, b: (ref.distill(a, b, tid, tl, None, T)["loss"] * gloss.double()).sum()  # noqa: E731
    h = 1e-5
    for _ in range(4):
        u = torch.randn((N, d), dtype=torch.float64, device=DEV, generator=g)
        diff = (f(x.double() + h * u, Wd) - f(x.double() - h * u, Wd)) / (2 * h)
        # second order is gone, third is h^2 of values near 1; the 64-bit loss rounds to 1e-13 / h
        assert abs(float((dx.double() * u).sum() - diff)) <= float((tx * u.abs()).sum()) + 1e-6
        u = torch.randn((Vd, d), dtype=torch.float64, device=DEV, generator=g)
        diff = (f(x, Wd.double() + h * u) - f(x, Wd.double() - h * u)) / (2 * h)
        assert abs(float((dW.double() * u).sum() - diff)) <= float((tW * u.abs()).sum()) + 1e-6


@pytest.mark.parametrize("N", [24, 160])
def test_teachers_that_leave_nothing_and_masked_places(N):
    g = gen(22)
    d, Vd, k = 128, 900, 8
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.05)
    tid, tl, _ = teacher_of(N, Vd, k, 0, g, empty=0.0)
    tid = (tid.long() % Vd).int()                        # every place has an id
    tid[0] = -1                                          # no teacher
    tl[1] = -math.inf                                    # no mass
    tl[2, 1:] = -math.inf                                # one alternative
    tid[3, 2:], tl[3, 2:] = -1, math.nan                 # what masked places hold has no say
    tid[4, 1:4] = tid[4, 0]                              # the same id four times
    tid[5] = tid[5, 0]                                   # ... and nothing else
    tl[6, 3:] = torch.finfo(torch.float32).min           # the type's lowest logit
    tl[7], tid[7, 0] = torch.finfo(torch.float32).min, -1
    tl[8, 4:], tid[9, 0] = -1e30, -1
    tl[9, 0] = math.inf
    loss, lse, z, dx, dW = step(x, Wd, tid, tl, None, 1.0, None)
    want = ref.distill(x, Wd, tid, torch.where(tid >= 0, tl, 0.0), None, 1.0)
    check_loss(loss, lse, want, 1.0, Vd)
    gx, gW, tx, tW = ref.grads(x, Wd, want, None, 1.0)
    within(dx, gx, tx, "dx")
    within(dW, gW, tW, "dWd")
    assert float(loss[0]) == 0 and float(loss[1]) == 0 and not bool(dx[:2].any())


@pytest.mark.parametrize("mapped", [False, True])
def test_teacher_ids_out_of_range(mapped):
    g = gen(23)
    N, d, Vd, k, V = 50, 64, 500, 4, 1300
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.1)
    tid, tl, t2d = teacher_of(N, Vd, k, V if mapped else 0, g, empty=0.0)
    bad = [3, 20, 49]
    broken = tid.clone()
    broken[3, 0], broken[20, 3], broken[49, 1] = (V if mapped else Vd), -2, -2 ** 31
    if mapped:
        t2d[:2] = torch.tensor([Vd, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        broken[7, 2], broken[8, 2] = 0, 1
        bad += [7, 8]
        broken[[i for i in range(N) if i not in bad]] = torch.where(broken < 2, -1, broken)[
            [i for i in range(N) if i not in bad]]
    good = broken.clone()
    good[bad] = -1                                       # such rows count like rows without a teacher
    ws, z = wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)
    loss, lse = wf.wf_draft_distill(x, Wd, broken, tl, ws, t2d=t2d, z=z)
    code, info = ws.device_error()
    assert code == BAD_DATA and info in bad
    dx, dW = wf.wf_draft_distill_grad(x, Wd, broken, tl, z, lse, ws, t2d=t2d)
    assert ws.device_error()[0] == BAD_DATA
    l2, s2, _, dx2, dW2 = step(x, Wd, good, tl, t2d, 1.0, None)
    ok = torch.ones(N, dtype=torch.bool, device=DEV)
    ok[bad] = False
    assert bool(torch.isnan(loss[~ok]).all()) and torch.equal(loss[ok], l2[ok]) and torch.equal(lse, s2)
    assert torch.equal(dx, dx2) and torch.equal(dW, dW2) and not bool(dx[~ok].any())


@pytest.mark.parametrize("N,d", [(33, 72), (300, 264)])
def test_distill_writes_its_outputs_only(N, d):
    g = gen(24)
    Vd, k = 1003, 5
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.05)
    tid, tl, _ = teacher_of(N, Vd, k, 0, g)
    out = dict(loss=Guarded((N,), torch.float32), lse=Guarded((N,), torch.float32))
    z = Guarded((N, 1016), torch.float32)
    z.t.fill_(7.5)
    dx, dW = Guarded((N, d), torch.bfloat16), Guarded((Vd, d), torch.bfloat16)
    ws = wf.DistillWorkspace(N, d, Vd, k)
    wf.wf_draft_distill(x, Wd, tid, tl, ws, z=z.t, **{n: o.t for n, o in out.items()})
    wf.wf_draft_distill_grad(x, Wd, tid, tl, z.t, out["lse"].t, ws, dx=dx.t, dWd=dW.t)
    want = ref.distill(x, Wd, tid, tl, None, 1.0)
    check_loss(out["loss"].t, out["lse"].t, want, 1.0, Vd)
    gx, gW, tx, tW = ref.grads(x, Wd, want, None, 1.0)
    within(dx.t, gx, tx, "dx")
    within(dW.t, gW, tW, "dWd")
    assert all(o.intact() for o in (*out.values(), z, dx, dW)) and bool((z.t[:, 1004:] == 7.5).all())


def test_distill_past_32_bit_offsets():
    """16,600 rows x 130,000 ids: 2.2e9 kept logits; the last rows lie past 2^31."""
    g = gen(25)
    N, d, Vd, k = 16600, 64, 130000, 3
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g, std=0.06)
    tid = torch.randint(0, Vd, (N, k), device=DEV, generator=g).int()
    tl = torch.randn((N, k), device=DEV, generator=g)
    gloss = torch.zeros(N, device=DEV)
    some = torch.tensor([0, 5, 9000, N - 300, N - 2, N - 1], device=DEV)
    gloss[some] = 1.0
    loss, lse, z, dx, dW = step(x, Wd, tid, tl, None, 1.0, gloss)
    xs, ts, ls = x[some].contiguous(), tid[some].contiguous(), tl[some].contiguous()
    want = ref.distill(xs, Wd, ts, ls, None, 1.0)
    check_loss(loss[some], lse[some], want, 1.0, Vd)
    gx, gW, tx, tW = ref.grads(xs, Wd, want, None, 1.0, rows=N)
    within(dx[some], gx, tx, "dx")
    within(dW, gW, tW, "dWd")
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[some] = False
    assert not bool(dx[rest].any())


@pytest.mark.parametrize("N,Vd", [(300, 3000), (300, 3001), (30, 1003)])
def test_distill_does_not_read_what_a_workspace_held(N, Vd):
    g = gen(26)
    d, k = 256, 6
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g)
    tid, tl, _ = teacher_of(N, Vd, k, 0, g)
    ws, z = wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)
    first = None
    for fill in (0x00, 0xFF, 0x7F):
        ws.buf[256:] = fill
        z.view(torch.uint8).fill_(fill)
        loss, lse = wf.wf_draft_distill(x, Wd, tid, tl, ws, z=z)
        ws.buf[256:] = fill                              # nothing passes between the calls but z and lse
        got = (loss, lse, *wf.wf_draft_distill_grad(x, Wd, tid, tl, z, lse, ws))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


# ------------------------------------------------------------------ as a program uses them
def _batch(g, N=260, d=256, V=9001, Vd=2000):
    h, W = ref.states(N, d, g), ref.head(V, d, g)
    x, Wd = ref.states(N, d, g), ref.head(Vd, d, g)
    d2t = torch.randperm(V, device=DEV, generator=g)[:Vd].sort().values.int()
    t2d = torch.full((V,), -1, dtype=torch.int32, device=DEV)
    t2d[d2t.long()] = torch.arange(Vd, dtype=torch.int32, device=DEV)
    return h, W, x, Wd, d2t, t2d


def test_a_drafter_is_distilled_from_the_target():
    """Teacher data from the target's head, two steps on the draft head, and the draft head's own candidates after."""
    g = gen(31)
    h, W, x, Wd, d2t, t2d = _batch(g)
    (N, d), V, Vd, k = x.shape, W.shape[0], Wd.shape[0], 16
    lws, dws, z = wf.LogprobsWorkspace(N, d, V, k=k), wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)
    gloss = torch.full((N,), 1.0 / N, device=DEV)
    for _ in range(2):
        best = wf.wf_lmhead_logprobs(h, W, lws, k=k)
        loss, lse = wf.wf_draft_distill(x, Wd, best.top_ids, best.top_logp, dws, t2d=t2d, z=z)
        dx, dW = wf.wf_draft_distill_grad(x, Wd, best.top_ids, best.top_logp, z, lse, dws, gloss=gloss, t2d=t2d)
        teach, _ = ref.logprobs(h, W, 1.0, None, k)
        assert torch.equal(best.top_ids, teach["top_ids"])
        want = ref.distill(x, Wd, best.top_ids, best.top_logp, t2d, 1.0)
        check_loss(loss, lse, want, 1.0, Vd)
        gx, gW, tx, tW = ref.grads(x, Wd, want, gloss, 1.0)
        within(dx, gx, tx, "dx")
        within(dW, gW, tW, "dWd")
        Wd = ref.grid(Wd.float() - 0.5 * dW.float(), 2.0 ** -11)
    ids, tids, vals = wf.wf_draft_topk(x, Wd, d2t, 4, wf.Workspace(0, N, 0, Vd, 4, d=d))
    order = torch.sort(x.double() @ Wd.double().T, dim=1, descending=True, stable=True).indices[:, :4].int()
    assert torch.equal(ids, order) and torch.equal(tids, d2t[order.long()])
    # an alternative of the draft head is a target id: the target's log-probability of it
    lp = wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(N, d, V, S=4), tok=tids)
    want, tol = ref.logprobs(h, W, 1.0, tids, 0)
    within(lp.logp, want["logp"], rows(tol["logp"], lp.logp), "logp")


def test_captured_steps_replay_on_new_inputs():
    """One graph of the whole step; and two graphs that share their workspaces, replayed in turn."""
    g = gen(32)
    h, W, x, Wd, d2t, t2d = _batch(g)
    (N, d), V, Vd, k = x.shape, W.shape[0], Wd.shape[0], 10
    lws, dws, z = wf.LogprobsWorkspace(N, d, V, k=k), wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)

    def run(h, x):
        best = wf.wf_lmhead_logprobs(h, W, lws, k=k, with_entropy=True)
        loss, lse = wf.wf_draft_distill(x, Wd, best.top_ids, best.top_logp, dws, t2d=t2d, z=z)
        return (*best[1:], loss, lse, *wf.wf_draft_distill_grad(x, Wd, best.top_ids, best.top_logp, z, lse, dws,
                                                                  t2d=t2d))

    ins = [(h.clone(), x.clone()) for _ in range(2)]
    run(*ins[0])
    graphs, outs = [], []
    for a in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(*a))
    for i in (0, 1, 0, 1):
        nh, nx = ref.states(N, d, g), ref.states(N, d, g)
        want = [t.clone() for t in run(nh, nx)]
        ins[i][0].copy_(nh)
        ins[i][1].copy_(nx)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


def test_two_streams_with_a_workspace_each():
    g = gen(33)
    h, W, x, Wd, d2t, t2d = _batch(g)
    (N, d), V, Vd, k = x.shape, W.shape[0], Wd.shape[0], 10
    work = [(wf.LogprobsWorkspace(N, d, V, k=k), wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd),
             torch.cuda.Stream()) for _ in range(2)]
    best = wf.wf_lmhead_logprobs(h, W, work[0][0], k=k)
    loss, lse = wf.wf_draft_distill(x, Wd, best.top_ids, best.top_logp, work[0][1], t2d=t2d, z=work[0][2])
    want = (*best[1:], loss, lse, *wf.wf_draft_distill_grad(x, Wd, best.top_ids, best.top_logp, work[0][2], lse,
                                                              work[0][1], t2d=t2d))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (lws, dws, z, s) in enumerate(work):
            with torch.cuda.stream(s):
                b = wf.wf_lmhead_logprobs(h, W, lws, k=k)
                lo, ls = wf.wf_draft_distill(x, Wd, b.top_ids, b.top_logp, dws, t2d=t2d, z=z)
                got[i].append((*b[1:], lo, ls, *wf.wf_draft_distill_grad(x, Wd, b.top_ids, b.top_logp, z, ls, dws,
                                                                       t2d=t2d)))
    torch.cuda.synchronize()
    for outs in got:
        for o in outs:
            assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(o, want))


def test_host_memory_is_refused():
    g = gen(34)
    h, W, x, Wd, d2t, t2d = _batch(g, N=8)
    ws = wf.LogprobsWorkspace(8, 256, 9001)
    with pytest.raises(ValueError):
        wf.wf_lmhead_logprobs(h.cpu(), W, ws)
    a = wf.LogprobsArgs(h.cpu().pin_memory().data_ptr(), W.data_ptr(), 8, 256, 9001, 1.0, None, 0, 0, None,
                        torch.empty(8, device=DEV).data_ptr())
    import ctypes
    assert wf.lib().wf_lmhead_logprobs(ctypes.byref(a), ws.ptr, ws.nbytes, None) == 1
    with pytest.raises(ValueError):
        wf.wf_lmhead_logprobs(h, W, wf.Workspace(8))
    with pytest.raises(wf.WfError):
        wf.wf_lmhead_logprobs(h, W, wf.LogprobsWorkspace(8, 256, 9001), k=17)
    with pytest.raises(wf.WfError):   # a workspace of fewer rows
        wf.wf_lmhead_logprobs(ref.states(3000, 256, g), W, ws)


def test_a_long_queue_of_steps_ends():
    """Hundreds of steps enqueued at once, no wait on the host between them: each kernel that takes whole SMs starts
    with nothing waiting beside it."""
    g = gen(35)
    h, W, x, Wd, d2t, t2d = _batch(g, N=300, Vd=9000, V=12001)
    (N, d), V, Vd, k = x.shape, W.shape[0], Wd.shape[0], 10
    lws, dws, z = wf.LogprobsWorkspace(N, d, V, k=k), wf.DistillWorkspace(N, d, Vd, k), wf.distill_logits(N, Vd)
    first = None
    for _ in range(400):
        best = wf.wf_lmhead_logprobs(h, W, lws, k=k)
        loss, lse = wf.wf_draft_distill(x, Wd, best.top_ids, best.top_logp, dws, t2d=t2d, z=z)
        got = (best.top_ids, loss, lse, *wf.wf_draft_distill_grad(x, Wd, best.top_ids, best.top_logp, z, lse, dws,
                                                                  t2d=t2d))
        first = first or [t.clone() for t in got]
    torch.cuda.synchronize()
    assert lws.device_error() == dws.device_error() == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(got, first))
