"""Plain 64-bit references of the heads' log-probabilities and of the draft head's distillation, and how far the
kernels' roundings may take an fp32 or bf16 result from them."""
import math

import torch

U = 2.0 ** -24          # half a step of fp32
BF = 2.0 ** -8          # half a step of bf16


def grid(x, step):
    """bf16 values of an 8-bit grid: sums of their products are exact in fp32 in any order."""
    return (torch.round(x / step).clamp(-127, 127) * step).to(torch.bfloat16)


def head(V, d, gen, on_grid=True, std=0.02):
    w = torch.randn((V, d), device=gen.device, generator=gen) * std
    return grid(w, 2.0 ** -11) if on_grid else w.to(torch.bfloat16)


def states(P, d, gen, on_grid=True):
    x = torch.randn((P, d), device=gen.device, generator=gen)
    return grid(x, 2.0 ** -5) if on_grid else x.to(torch.bfloat16)


def logits(x, W, T):
    return (x.double() @ W.double().T) / T


def logit_error(x, W, T, on_grid):
    """Most that an fp32 sum of a logit is off: nothing on the grid, else d steps on the sum of magnitudes."""
    if on_grid:
        return torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    return ((x.double().abs() @ W.double().abs().T).amax(1)) * 2 * x.shape[1] * U / T


def sum_error(V):
    """Relative error of a sum over V exponentials: the exponential's own 2 units in the last place, and at most a
    rounding for each group of 32 columns, each of the four partial sums' 8 terms and each merge of 160 states."""
    return (V / 32 + 8 + 3 + 160 + 8) * U


def logprobs(x, W, T, tok, k, on_grid=True):
    """Results of wf_lmhead_logprobs in 64 bits, and the tolerances of lse, H and of a log-probability."""
    raw = x.double() @ W.double().T
    z = raw / T
    lse = torch.logsumexp(z, 1)
    lq = z - lse[:, None]
    q = lq.exp()
    H = torch.special.entr(q).sum(1)
    logp = None
    if tok is not None:
        t2 = tok.reshape(tok.shape[0], -1).long()
        logp = torch.where(t2 >= 0, torch.gather(lq, 1, t2.clamp(min=0)), 0.0).reshape(tok.shape)
    top_ids = top_logp = None
    if k:
        order = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :k]
        top_ids, top_logp = order.int(), torch.gather(lq, 1, order)
    el = logit_error(x, W, T, on_grid)
    # 1/T, log2 e and their product are rounded (3 U of a logit), then the exponent's fma and reference: 2 more
    ez = el + 5 * U * z.abs().amax(1)
    es = sum_error(W.shape[0])
    spread = (q * (z - (q * z).sum(1, keepdim=True)).abs()).sum(1)
    mean = (q * (z.amax(1, keepdim=True) - z)).sum(1)
    tol = dict(lse=2 * ez + es + 4 * U * lse.abs(), logp=2 * ez + es + 4 * U * lq.abs().amax(1),
               H=2 * ez * spread + es * (1 + 2 * mean) + 8 * U * (1 + H + mean))
    return dict(logp=logp, lse=lse, H=H, top_ids=top_ids, top_logp=top_logp), tol


def teacher(tid, tlogit, t2d, T, Vd):
    """[N, k] draft ids (0 where not kept) and probabilities (0 there), [N] kept any."""
    ids = tid.long()
    if t2d is not None:
        ids = torch.where(ids >= 0, t2d.long()[ids.clamp(min=0)], -1)
    keep = (ids >= 0) & (tlogit != -math.inf)
    t = torch.where(keep, tlogit.double() / T, -math.inf)
    some = keep.any(1)
    t = torch.where(some[:, None], t, 0.0)
    p = torch.where(keep & some[:, None], torch.softmax(t, 1), 0.0)
    return torch.where(keep, ids, 0), p, some


def distill(x, Wd, tid, tlogit, t2d, T):
    z = logits(x, Wd, T)
    lse = torch.logsumexp(z, 1)
    ids, p, some = teacher(tid, tlogit, t2d, T, Wd.shape[0])
    lq = torch.gather(z, 1, ids) - lse[:, None]
    loss = torch.where(p > 0, p * (torch.log(torch.where(p > 0, p, 1.0)) - lq), 0.0).sum(1)
    return dict(z=z, lse=lse, loss=loss, ids=ids, p=p, some=some)


def grads(x, Wd, r, gloss, T, rows=None):
    """dx, dWd in 64 bits and their tolerances, element by element: G is off by half a step of bf16 (up to 128 rows: by
    half a step of what half a step leaves; rows: of the call, where x holds some of them) and by what z, lse and p are off, the products by their fp32 sums, the
    results by another half step of bf16."""
    N = x.shape[0]
    g = torch.ones(N, dtype=torch.float64, device=x.device) if gloss is None else gloss.double()
    gs = torch.where(r["some"], g / T, 0.0)[:, None]
    q = torch.exp(r["z"] - r["lse"][:, None])
    pt = torch.zeros_like(q).scatter_add_(1, r["ids"], r["p"])
    G = gs * (q - pt)
    # z and lse in fp32, off by what the forward call's tolerances say; the exponential; p's softmax
    ez = 8 * U * (r["z"].abs().amax(1, keepdim=True) + r["lse"].abs()[:, None]) + sum_error(Wd.shape[0])
    eG = (BF if (rows or N) > 128 else BF * BF) * G.abs() + gs.abs() * (q * (ez + 8 * U) + pt * (80 * U + 4 * U * 40))
    W, X = Wd.double(), x.double()
    dx, dW = G @ W, G.T @ X
    tol_x = (1 + BF) * (eG @ W.abs() + 4 * Wd.shape[0] * U * (G.abs() @ W.abs())) + BF * dx.abs() + 1e-38
    tol_W = (1 + BF) * (eG.T @ X.abs() + 4 * N * U * (G.abs().T @ X.abs())) + BF * dW.abs() + 1e-38
    return dx, dW, tol_x, tol_W
