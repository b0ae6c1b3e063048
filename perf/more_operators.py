"""Workloads of the heads' log-probabilities and of the draft head's distillation.

Each case is one pass: `logprobs` (the log-probabilities of given tokens under the target head, with the entropy and the
top alternatives), `loss` (the distillation loss of the draft head against a teacher's top logits, as an evaluation
reads it) and `step` (the loss and its gradients with respect to the drafter's states and the draft head).  With `own`
false `run` computes the plain form in torch.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a tiny head: nothing but latency
        dict(name="tiny_rows", op="logprobs", P=17, d=256, V=8192, S=1, k=3, T=1.0),
        # the token that one user's step sampled, with five alternatives
        dict(name="one_token", op="logprobs", P=1, d=2560, V=151936, S=1, k=5, T=0.7),
        # a verified block: the drafted tokens' log-probabilities
        dict(name="chain_rows", op="logprobs", P=17, d=2560, V=151936, S=1, k=0, T=1.0),
        # a verified tree: each row's children and ten alternatives
        dict(name="tree_rows", op="logprobs", P=61, d=2560, V=151936, S=10, k=10, T=1.0),
        # the rows of a mixed batch of 32 rounds
        dict(name="mixed_rows", op="logprobs", P=1248, d=2560, V=151936, S=1, k=10, T=1.0),
        # a long prompt scored as a teacher's data are made: sixteen alternatives a row
        dict(name="prompt_rows", op="logprobs", P=3967, d=2560, V=151936, S=1, k=16, T=1.0),
        # the loss of a few rows over a tiny head
        dict(name="loss_tiny", op="loss", N=16, d=256, Vd=1000, k=4, V=0, T=1.0),
        # an evaluation batch
        dict(name="loss_batch", op="loss", N=2048, d=2560, Vd=32000, k=10, V=151936, T=1.0),
        # a step on one short sequence: the head's weights outweigh the rows
        dict(name="step_short", op="step", N=64, d=2560, Vd=32000, k=10, V=151936, T=1.0),
        # odd sizes, a softened teacher
        dict(name="step_odd", op="step", N=777, d=1024, Vd=10007, k=16, V=50257, T=2.0),
        # a teacher whose 64 best were kept, ids of the draft vocabulary itself
        dict(name="step_wide_teacher", op="step", N=1500, d=2048, Vd=32000, k=64, V=0, T=1.0),
        # a full training batch
        dict(name="step_batch", op="step", N=4096, d=2560, Vd=32000, k=10, V=151936, T=1.0),
    ]


MOST = 3967 * 151936 * 2560          # products of the largest listed case


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["logprobs", "logprobs", "loss", "step", "step"])
    d = rng.choice([256, 512, 1000, 1024, 2048, 2560, 4096])
    T = rng.choice([0.5, 0.7, 1.0, 1.0, 2.0])
    if op == "logprobs":
        V = _log_int(rng, 1000, 151936)
        return dict(op=op, P=_log_int(rng, 1, max(1, min(4096, MOST // (V * d)))), d=d, V=V,
                    S=rng.choice([0, 1, 1, 4, 16]), k=rng.choice([0, 1, 5, 10, 16]), T=T)
    Vd = _log_int(rng, 1000, 65536)
    most = min(4096, MOST // (Vd * d) // (3 if op == "step" else 1))
    return dict(op=op, N=_log_int(rng, 1, max(1, most)), d=d, Vd=Vd, k=rng.choice([1, 4, 10, 16, 64]),
                V=rng.choice([0, 2 * Vd, 5 * Vd + 3]), T=T)


def work(case):
    d, k = case["d"], case["k"]
    if case["op"] == "logprobs":
        P, V, S = case["P"], case["V"], case["S"]
        return {"bytes": 2 * (P + V) * d + 8 * P * S + 8 * P + 8 * P * k, "flops": 2 * P * V * d}
    N, Vd = case["N"], case["Vd"]
    loss = 2 * (N + Vd) * d + 8 * N * k + 8 * N + 4 * case["V"]
    if case["op"] == "loss":
        return {"bytes": loss, "flops": 2 * N * Vd * d}
    return {"bytes": loss + 4 * N + 2 * (N + Vd) * d, "flops": 6 * N * Vd * d}


# ------------------------------------------------------------------ inputs
W_STEP, H_STEP = 2.0 ** -11, 2.0 ** -5


def _grid(x, step):
    """Values of an 8-bit symmetric grid, as quantised weights and states hold them: every order of summation gives the
    same logits, so equal and nearly equal alternatives rank the same for everyone."""
    return (torch.round(x / step).clamp_(-127, 127) * step).to(torch.bfloat16)


def _weights(rows, d, gen):
    return _grid(torch.randn((rows, d), device=DEV, generator=gen).mul_(0.02), W_STEP)


def _states(W, rows, T, gen):
    """Final hidden states: noise, and towards three tokens each, up to where the first has most of the probability at
    temperature T: some rows are sure of their token and others are not.  And those tokens."""
    n, (V, d) = rows, W.shape
    pick = torch.randint(0, V, (n, 3), device=DEV, generator=gen)
    sure = torch.rand((n, 3), device=DEV, generator=gen) * torch.tensor([1.0, 0.8, 0.6], device=DEV)
    x = torch.randn((n, d), device=DEV, generator=gen)
    for j in range(3):
        # W's rows have length 0.02 sqrt d: at most a logit of T log V
        x += sure[:, j:j + 1] * W[pick[:, j]].float() * (T * math.log(V) / (0.02 ** 2 * d))
    return _grid(x, H_STEP), pick


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * int(seed) + 29)
    d, k = case["d"], case["k"]
    s = dict(case=case)
    if case["op"] == "logprobs":
        P, V, S = case["P"], case["V"], case["S"]
        s["W"] = _weights(V, d, gen)
        s["hidden"], pick = _states(s["W"], P, case["T"], gen)
        s["tok"] = None
        if S:
            tok = torch.randint(0, V, (P, S), device=DEV, generator=gen)
            m = min(S, 3)
            tok[:, :m] = pick[:, :m]
            if S > 1:                                   # a row with fewer children than columns
                tok[torch.rand((P, S), device=DEV, generator=gen) < 0.2] = -1
            s["tok"] = tok.to(torch.int32)
        if own:
            from speculative_decoding_verify_lm_gb300 import wf
            s["ws"] = wf.LogprobsWorkspace(P, d, V, S=S, k=k)
        return s
    N, Vd, V = case["N"], case["Vd"], case["V"]
    s["Wd"] = _weights(Vd, d, gen)
    s["x"], pick = _states(s["Wd"], N, case["T"], gen)
    # the teacher's best: distinct ids, the student's own among them, logits falling from the first
    ids = (pick[:, :1] + torch.arange(k, device=DEV)[None] * (1 + torch.randint(0, max(1, (Vd - 1) // k), (N, 1),
                                                                                  device=DEV, generator=gen))) % Vd
    fall = torch.empty((N, k), device=DEV).exponential_(1.0 / 0.6, generator=gen)
    s["tlogit"] = 18.0 - torch.cumsum(fall, 1)
    s["t2d"] = None
    if V:
        d2t = torch.randperm(V, device=DEV, generator=gen)[:Vd]
        s["t2d"] = torch.full((V,), -1, dtype=torch.int32, device=DEV)
        s["t2d"][d2t] = torch.arange(Vd, dtype=torch.int32, device=DEV)
        # one in six of the teacher's alternatives has no draft id
        ids = torch.where(torch.rand((N, k), device=DEV, generator=gen) < 1 / 6,
                          torch.randint(0, V, (N, k), device=DEV, generator=gen), d2t[ids])
    empty = torch.rand((N, 1), device=DEV, generator=gen) < 0.05            # rows without a teacher
    s["tid"] = torch.where(empty, -1, ids).to(torch.int32)
    if case["op"] == "step":
        # a weight for each row: the mean over the rows that count, and positions weighed differently
        s["gloss"] = torch.rand(N, device=DEV, generator=gen) / N
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        s["ws"] = wf.DistillWorkspace(N, d, Vd, k)
        if case["op"] == "step":
            s["z"] = wf.distill_logits(N, Vd)
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    return {"logprobs": _logprobs, "loss": _loss, "step": _step}[s["case"]["op"]](s)


def _logprobs(s):
    c = s["case"]
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        r = wf.wf_lmhead_logprobs(s["hidden"], s["W"], s["ws"], tok=s["tok"], k=c["k"], temperature=c["T"],
                                  with_entropy=True)
        return {"logp": r.logp, "lse": r.lse, "H": r.H, "top_ids": r.top_ids, "top_logp": r.top_logp}
    z = s["hidden"].float() @ s["W"].float().T
    top_ids = top_logp = None
    if c["k"]:
        # equal logits rank by id: the order of the bits, then the lower id
        bits = z.view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * 2 ** 32
        key -= torch.arange(c["V"], device=DEV)
        best = torch.topk(key, c["k"], dim=1).values
        del bits, key
        top = -best % 2 ** 32
        top_ids = top.to(torch.int32)
    z = z / c["T"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    logs = torch.log(total)
    H = logs[:, 0] - (e * (z - m)).sum(1) / total[:, 0]
    if c["k"]:
        top_logp = torch.gather(z, 1, top) - m - logs
    logp = None
    if s["tok"] is not None:
        tok = s["tok"].long()
        logp = torch.where(tok >= 0, torch.gather(z, 1, tok.clamp(min=0)) - m - logs, 0.0)
    return {"logp": logp, "lse": (m + logs)[:, 0], "H": H, "top_ids": top_ids, "top_logp": top_logp}


def _teacher(s):
    """Draft ids (0 where there is none), probabilities (0 there) and which rows have any."""
    tid = s["tid"].long()
    ids = tid if s["t2d"] is None else torch.where(tid >= 0, s["t2d"].long()[tid.clamp(min=0)], -1)
    there = ids >= 0
    t = torch.where(there, s["tlogit"] / s["case"]["T"], -math.inf)
    some = there.any(1, keepdim=True)
    p = torch.where(there, torch.exp(t - torch.where(some, t.amax(1, keepdim=True), 0.0)), 0.0)
    p = p / torch.where(some, p.sum(1, keepdim=True), 1.0)
    return ids.clamp(min=0), p, some[:, 0]


def _forward(s):
    z = s["x"].float() @ s["Wd"].float().T / s["case"]["T"]
    m = z.amax(1, keepdim=True)
    logs = torch.log(torch.exp(z - m).sum(1, keepdim=True))
    ids, p, some = _teacher(s)
    logq = torch.gather(z, 1, ids) - m - logs
    loss = torch.where(p > 0, p * (torch.log(torch.where(p > 0, p, 1.0)) - logq), 0.0).sum(1)
    return z, (m + logs)[:, 0], ids, p, some, loss


def _loss(s):
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        loss, lse = wf.wf_draft_distill(s["x"], s["Wd"], s["tid"], s["tlogit"], s["ws"], t2d=s["t2d"],
                                        temperature=s["case"]["T"])
        return {"loss": loss, "lse": lse}
    _, lse, _, _, _, loss = _forward(s)
    return {"loss": loss, "lse": lse}


def _step(s):
    T = s["case"]["T"]
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        loss, lse = wf.wf_draft_distill(s["x"], s["Wd"], s["tid"], s["tlogit"], s["ws"], t2d=s["t2d"], temperature=T,
                                        z=s["z"])
        dx, dWd = wf.wf_draft_distill_grad(s["x"], s["Wd"], s["tid"], s["tlogit"], s["z"], lse, s["ws"],
                                           gloss=s["gloss"], t2d=s["t2d"], temperature=T)
        return {"loss": loss, "lse": lse, "dx": dx, "dWd": dWd}
    z, lse, ids, p, some, loss = _forward(s)
    q = torch.exp(z - lse[:, None])
    G = q.scatter_add_(1, ids, -p) * torch.where(some, s["gloss"] / T, 0.0)[:, None]
    dx = G @ s["Wd"].float()
    dWd = G.T @ s["x"].float()
    return {"loss": loss, "lse": lse, "dx": dx.to(torch.bfloat16), "dWd": dWd.to(torch.bfloat16)}


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_logprobs(case, s) if case["op"] == "logprobs" else _exact_distill(case, s)


def _exact_logprobs(case, s):
    W, parts = s["W"].double(), []
    for r in range(0, case["P"], 512):
        z = torch.einsum("pd,vd->pv", s["hidden"][r:r + 512].double(), W) / case["T"]
        logq = torch.log_softmax(z, 1)
        part = {"logp": None, "lse": torch.logsumexp(z, 1), "H": torch.special.entr(logq.exp()).sum(1), "top_ids": None,
                "top_logp": None}
        if s["tok"] is not None:
            part["logp"] = torch.zeros_like(s["tok"][r:r + 512], dtype=torch.float64)
            row, col = torch.nonzero(s["tok"][r:r + 512] >= 0, as_tuple=True)
            part["logp"][row, col] = logq[row, s["tok"][r:r + 512][row, col].long()]
        if case["k"]:
            best = torch.sort(logq, dim=1, descending=True, stable=True)
            part["top_ids"] = best.indices[:, :case["k"]].to(torch.int32)
            part["top_logp"] = best.values[:, :case["k"]]
        parts.append(part)
    return {name: None if parts[0][name] is None else torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_distill(case, s):
    N, T, W = case["N"], case["T"], s["Wd"].double()
    out = {"loss": [], "lse": [], "dx": []}
    dW = torch.zeros_like(W) if case["op"] == "step" else None
    for r in range(0, N, 1024):
        x = s["x"][r:r + 1024].double()
        n = x.shape[0]
        z = torch.einsum("nd,vd->nv", x, W) / T
        logq = torch.log_softmax(z, 1)
        # the teacher's distribution over the whole draft vocabulary
        p = torch.zeros_like(z)
        tid = s["tid"][r:r + n].long()
        row, col = torch.nonzero(tid >= 0, as_tuple=True)
        ids = tid[row, col]
        if s["t2d"] is not None:
            ids = s["t2d"].long()[ids]
            row, col, ids = row[ids >= 0], col[ids >= 0], ids[ids >= 0]
        p.index_put_((row, ids), torch.exp(s["tlogit"][r:r + n].double()[row, col] / T), accumulate=True)
        mass = p.sum(1, keepdim=True)
        p = torch.where(mass > 0, p / mass, 0.0)
        # entries that name the same id count as one here; the kept ids of a row are distinct but for chance
        weight = torch.exp(s["tlogit"][r:r + n].double()[row, col] / T) / mass[row, 0]
        loss = torch.zeros(n, dtype=torch.float64, device=DEV)
        loss.index_add_(0, row, weight * (torch.log(weight) - logq[row, ids]))
        out["loss"].append(loss)
        out["lse"].append(torch.logsumexp(z, 1))
        if dW is not None:
            G = (logq.exp() - p) * (torch.where(mass[:, 0] > 0, s["gloss"][r:r + n].double(), 0.0) / T)[:, None]
            out["dx"].append(torch.einsum("nv,vd->nd", G, W))
            dW += torch.einsum("nv,nd->vd", G, x)
    got = {"loss": torch.cat(out["loss"]), "lse": torch.cat(out["lse"])}
    if dW is not None:
        got["dx"], got["dWd"] = torch.cat(out["dx"]), dW
    return got
