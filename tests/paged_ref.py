"""The paged cache's operators in plain numpy, 64 bits, one sequence after
another: what the GPU tests compare with.  Types: caches are float64 arrays of
the values they hold (a bf16 or e4m3 value is exact in fp64)."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16 = 2.0 ** -8      # half a step, relative
FP16 = 2.0 ** -11
FP32 = 2.0 ** -24


class Case:
    """A cache of B sequences with every position that no sequence owns poisoned (NaN), and a round's rows."""

    def __init__(self, seed, lens, rows, H, G, D, ps, kv="bf16", kinds=None, layers=1, layer=0, extra_rows=0,
                 first_row=0, slack=3, spread=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.rows = rng, list(lens), list(rows)
        self.H, self.G, self.D, self.ps, self.kv, self.layers, self.layer = H, G, D, ps, kv, layers, layer
        self.B = B = len(lens)
        self.kinds = [0] * B if kinds is None else list(kinds)
        need = [-(-(n + r) // ps) for n, r in zip(lens, rows)]
        self.num_pages = sum(need) + slack
        self.max_pages = max(max(need), 1) + 1
        order = rng.permutation(self.num_pages)
        self.table = np.full((B, self.max_pages), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        shape = (layers, self.num_pages, ps, G, D)
        self.k_scale = self.v_scale = None
        K = torch.full(shape, float("nan"))
        V = torch.full(shape, float("nan"))
        if kv == "e4m3":
            self.k_scale = rng.uniform(0.3, 3.0, (layers, G)).astype(np.float32)
            self.v_scale = rng.uniform(0.3, 3.0, (layers, G)).astype(np.float32)
        self.dtype = torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16
        for b in range(B):
            T = self.lens[b] + self.rows[b]
            pg, at = self.table[b, np.arange(T) // ps], np.arange(T) % ps
            K[:, pg, at] = torch.from_numpy(rng.standard_normal((layers, T, G, D)) * spread).float()
            V[:, pg, at] = torch.from_numpy(rng.standard_normal((layers, T, G, D))).float()
        self.K, self.V = K.to(self.dtype), V.to(self.dtype)
        self.pos_off = np.cumsum([first_row] + self.rows).astype(np.int32)
        self.P = int(self.pos_off[-1]) + extra_rows
        self.q = torch.from_numpy(rng.standard_normal((self.P, H, D))).to(torch.bfloat16)
        self.node_off = np.cumsum([0] + [max(r - 1, 0) for r in self.rows]).astype(np.int32)
        par = []
        for b in range(B):
            for i in range(self.rows[b] - 1):
                par.append(int(rng.integers(max(-1, i - 9), i)) if self.kinds[b] else i - 1)
        self.parent = np.array(par if par else [0], np.int32)

    def sees(self, b):
        """[rows, rows] bool: row i sees row j of the round."""
        n = self.rows[b]
        m = np.zeros((n, n), bool)
        for i in range(n):
            if not self.kinds[b]:
                m[i, :i + 1] = True
                continue
            j = i
            while j > 0:
                m[i, j] = True
                j = 1 + int(self.parent[self.node_off[b] + j - 1])
            m[i, 0] = True
        return m

    def dense(self, b, g, which):
        """[T, D] float64 keys or values of a sequence, scaled."""
        pool = (self.K if which == "K" else self.V)[self.layer]
        t = np.arange(self.lens[b] + self.rows[b])
        x = pool.float()[self.table[b, t // self.ps], t % self.ps, g].numpy().astype(np.float64)
        sc = self.k_scale if which == "K" else self.v_scale
        return x if sc is None else x * float(sc[self.layer, g])


def attention(c: Case, scale):
    """-> out, lse, tolerance of out, tolerance of lse ([P, H, D] / [P, H]; NaN where no sequence has the row).

    Rounding points: scores in fp32 (D products: D 2^-24 sum |q k| scale; for an
    e4m3 cache also the fp16 query, off by at most 2^-25 of the row's largest
    element), e^x (2^-21), the probability's rounding to the 16-bit type, the
    fp32 sums over T positions, and the output's rounding to bf16."""
    H, G, D = c.H, c.G, c.D
    hq = H // G
    out = np.full((c.P, H, D), np.nan)
    lse = np.full((c.P, H), np.nan)
    tol = np.zeros((c.P, H, D))
    tol_l = np.zeros((c.P, H))
    p16 = BF16 if c.kv == "bf16" else FP16
    q = c.q.float().numpy().astype(np.float64)
    for b in range(c.B):
        n, L = c.rows[b], c.lens[b]
        if n == 0:
            continue
        see = np.concatenate([np.ones((n, L), bool), c.sees(b)], 1)
        T = L + n
        r0 = int(c.pos_off[b])
        for g in range(G):
            K, V = c.dense(b, g, "K"), c.dense(b, g, "V")
            for h in range(g * hq, (g + 1) * hq):
                x = q[r0:r0 + n, h]
                for i in range(n):
                    k, v = K[see[i]], V[see[i]]
                    s = scale * (k @ x[i])
                    top = s.max()
                    w = np.exp(s - top)
                    w, total = w / w.sum(), w.sum()
                    o = w @ v
                    ds = scale * (D * FP32 * (np.abs(k) @ np.abs(x[i]))).max() + 2.0 ** -22 * np.abs(s).max()
                    if c.kv == "e4m3":
                        ds += scale * 2.0 ** -25 * np.abs(x[i]).max() * np.abs(k).sum(1).max()
                    mass = w @ np.abs(v)
                    rel = p16 + 2 * ds + 2.0 ** -20 + 2 * T * FP32
                    if c.kv == "e4m3":      # probabilities below 2^-33 of the largest round to fp16's least step
                        mass = mass + T * 2.0 ** -22 * np.abs(v).max(0)
                    out[r0 + i, h] = o
                    tol[r0 + i, h] = rel * mass + BF16 * (np.abs(o) + rel * mass)
                    lse[r0 + i, h] = top + math.log(total)
                    tol_l[r0 + i, h] = 2 * ds + 2.0 ** -20 + T * FP32 + 2.0 ** -22 * abs(lse[r0 + i, h])
    return out, lse, tol, tol_l


# ------------------------------------------------------------------ pages
def reserve(table, ref, lens, rows, ps):
    """In order of the sequences.  -> (table, ref, added, copies [(from, to)])."""
    table, ref = table.copy(), ref.copy()
    B, width = table.shape
    plan, free = [], [p for p in range(len(ref)) if ref[p] == 0]
    count = ref.copy()      # references as they would be if everything fitted
    taken, added, copies, out_of = 0, [], [], False
    for b in range(B):
        n, r = int(lens[b]), int(rows[b])
        ok = n >= 0 and r >= 0 and n + r <= width * ps
        todo = []
        if ok and r > 0:
            for j in range(n // ps, -(-(n + r) // ps)):
                e = int(table[b, j])
                if e < -1 or e >= len(ref) or (j == n // ps and n % ps and e < 0):
                    ok = False
                    break
                if e < 0:
                    todo.append((j, None))
                elif count[e] > 1:
                    todo.append((j, e))
        if not ok:
            added.append(-1)
            continue
        for _, e in todo:
            if e is not None:
                count[e] -= 1
        if out_of or taken + len(todo) > len(free):
            out_of = True
            added.append(-1)
            continue
        for j, e in todo:
            p = free[taken]
            taken += 1
            ref[p] = 1
            if e is not None:
                ref[e] -= 1
                if j == n // ps and n % ps:
                    copies.append((e, p))
            table[b, j] = p
        added.append(len(todo))
    return table, ref, np.array(added, np.int32), copies


def fork(table, ref, lens, src, dst, ps):
    table, ref, lens = table.copy(), ref.copy(), lens.copy()
    B, width = table.shape
    bad = []
    t0, l0 = table.copy(), lens.copy()
    for i, (a, d) in enumerate(zip(src, dst)):
        ok = 0 <= a < B and 0 <= d < B and list(dst).count(d) == 1 and d not in list(src)
        if ok:
            n = -(-int(l0[a]) // ps)
            ok = l0[a] >= 0 and n <= width and (t0[d] < 0).all() and (t0[a, :n] >= 0).all() and \
                (t0[a, :n] < len(ref)).all()
        if not ok:
            bad.append(i)
            continue
        table[d] = -1
        table[d, :n] = t0[a, :n]
        for p in t0[a, :n]:
            ref[p] += 1
        lens[d] = l0[a]
    return table, ref, lens, bad


def trim(table, ref, lens, ps):
    table, ref = table.copy(), ref.copy()
    for b in range(table.shape[0]):
        if lens[b] < 0:
            continue
        for j in range(-(-int(lens[b]) // ps), table.shape[1]):
            p = table[b, j]
            if p >= 0:
                ref[p] -= 1
            table[b, j] = -1
    return table, ref


def nearest_e4m3(x):
    """The nearest e4m3 value (ties to even), saturating; x float64, no NaN."""
    a = np.minimum(np.abs(x), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = np.ldexp(1.0, (e - 3).astype(int))
    return np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)
