"""Workloads of the paged key-value cache's operators.

Each case is one call (or, for the page bookkeeping, one step's three calls) on a cache whose keys and values
live in pages: `attention` (single new tokens, drafted chains and trees over their prefix), `append` (a round's
keys and values into their pages), `compact` (the accepted path's rows moved up in every layer) and `pages`
(trim, fork and reserve with copy on write).  With `own` false `run` computes the plain form in torch.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the drafter's next token for one user: nothing but latency (drafter geometry: 32 heads over 8, width 80)
        dict(name="one_token_drafter", op="attention", B=1, form="one", R=1, lo=2048, hi=2048, H=32, G=8, D=80, ps=16,
             kv="bf16"),
        # one user deep in a long document
        dict(name="one_token_long", op="attention", B=1, form="one", R=1, lo=131000, hi=131000, H=32, G=8, D=128,
             ps=64, kv="bf16"),
        # a served batch of very different lengths
        dict(name="one_token_ragged", op="attention", B=64, form="one", R=1, lo=100, hi=16384, H=32, G=8, D=128,
             ps=16, kv="bf16"),
        # a larger batch on an 8-bit cache
        dict(name="one_token_e4m3", op="attention", B=128, form="one", R=1, lo=2000, hi=6000, H=32, G=8, D=128, ps=32,
             kv="e4m3"),
        # a 60-node tree of one user: the verified rows' attention at batch 1
        dict(name="tree_one_user", op="attention", B=1, form="tree", R=61, lo=2048, hi=2048, H=32, G=8, D=128, ps=16,
             kv="bf16"),
        # the mixed batch: chains of 16 and trees of 60 drafted tokens
        dict(name="mixed_batch", op="attention", B=32, form="mixed", R=61, lo=1500, hi=6000, H=32, G=8, D=128, ps=16,
             kv="bf16"),
        # the trees of a full batch enter the cache
        dict(name="append_trees", op="append", B=256, form="tree", R=61, lo=5, hi=90, G=8, D=128, ps=16, kv="bf16"),
        # one chain enters an 8-bit cache
        dict(name="append_chain_e4m3", op="append", B=1, form="chain", R=17, lo=1000, hi=1000, G=8, D=80, ps=16,
             kv="e4m3"),
        # after a round of one user: a few rows move in every layer
        dict(name="compact_one_user", op="compact", B=1, form="tree", R=61, lo=333, hi=333, G=8, D=128, ps=16,
             kv="bf16", layers=32),
        # after a round of the mixed batch's size
        dict(name="compact_batch", op="compact", B=48, form="tree", R=61, lo=20, hi=60, G=8, D=128, ps=16, kv="bf16",
             layers=32),
        # three continuations of one prompt begin
        dict(name="fork_one_prompt", op="pages", B=1, kids=3, lo=777, hi=777, G=8, D=80, ps=16, kv="bf16", layers=1),
        # four continuations of each of sixteen prompts begin, on a deep model
        dict(name="fork_batch", op="pages", B=16, kids=4, lo=100, hi=500, G=8, D=128, ps=16, kv="bf16", layers=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["attention", "attention", "attention", "append", "compact", "pages"])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    G, hq = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    D, ps = rng.choice([64, 80, 96, 128]), rng.choice([8, 16, 32, 64, 128])
    if op == "attention":
        form = rng.choice(["one", "one", "chain", "tree", "mixed"])
        R = 1 if form == "one" else _log_int(rng, 2, 150)
        B = _log_int(rng, 1, 128 if form == "one" else 32)
        # no more keys read, and no more products, than the largest listed cases have
        most = min(131000, 800000000 // (4 * B * G * D))
        if form != "one":
            most = min(6000, most, 60000000000 // (4 * B * R * G * hq * D))
        hi = _log_int(rng, min(64, most), most)
        return dict(op=op, B=B, form=form, R=R, lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, H=G * hq, G=G, D=D,
                    ps=ps, kv=kv)
    if op == "append":
        return dict(op=op, B=_log_int(rng, 1, 256), form=rng.choice(["chain", "tree", "mixed"]),
                    R=_log_int(rng, 1, 61), lo=1, hi=_log_int(rng, 2, 300), G=G, D=D, ps=ps, kv=kv)
    if op == "compact":
        return dict(op=op, B=_log_int(rng, 1, 48), form=rng.choice(["tree", "mixed"]),
                    R=_log_int(rng, 8, 61), lo=1, hi=_log_int(rng, 2, 60), G=G, D=D, ps=ps, kv=kv,
                    layers=_log_int(rng, 1, 32))
    return dict(op=op, B=_log_int(rng, 1, 16), kids=rng.choice([1, 2, 3, 4]), lo=50, hi=_log_int(rng, 51, 400), G=G,
                D=D, ps=rng.choice([8, 16, 32]), kv=kv, layers=_log_int(rng, 1, 24))


# ------------------------------------------------------------------ the shape of a case
def _plan(case):
    """Lengths, row counts, kinds, parents and accepted paths: fixed by the case, not by the seed."""
    rng = random.Random("|".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [_log_int(rng, lo, hi) for _ in range(B)]
    form, R = case.get("form", "one"), case.get("R", 1)
    rows, kinds = [], []
    for b in range(B):
        tree = form == "tree" or (form == "mixed" and b % 2 == 1)
        kinds.append(1 if tree else 0)
        rows.append(min(R, 17) if form == "mixed" and not tree else R)
    pos_off, node_off, parent, path, n_accept = [0], [0], [], [], []
    depth_max = 16
    for b in range(B):
        n = rows[b] - 1
        par = [i - 1 if not kinds[b] else rng.randint(max(-1, i - 12), i - 1) for i in range(n)]
        parent += par
        pos_off.append(pos_off[-1] + rows[b])
        node_off.append(node_off[-1] + n)
        if n:
            i, way = rng.randrange(n // 2, n), []
            while i >= 0:
                way.append(i)
                i = par[i]
            way = way[::-1][:depth_max]
            if not kinds[b]:
                way = way[:rng.randint(0, depth_max)]
        else:
            way = []
        n_accept.append(len(way))
        path.append(way + [-1] * (depth_max - len(way)))
    return dict(lens=lens, rows=rows, kinds=kinds, pos_off=pos_off, node_off=node_off, parent=parent, path=path,
                n_accept=n_accept)


def _visible(p):
    """Keys that all rows of the case see together."""
    total = 0
    for b, n in enumerate(p["rows"]):
        depth = []
        for i in range(n - 1):
            q = p["parent"][p["node_off"][b] + i]
            depth.append(1 if q < 0 else depth[q] + 1)
        total += n * (p["lens"][b] + 1) + sum(depth)
    return total


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    p = _plan(case)
    e = 2 if case["kv"] == "bf16" else 1
    row = case["G"] * case["D"]                    # elements of one position's keys
    if case["op"] == "attention":
        P, H = sum(p["rows"]), case["H"]
        T = sum(a + b for a, b in zip(p["lens"], p["rows"]))
        return {"bytes": 2 * T * row * e + 4 * P * H * case["D"] + 4 * P * H,
                "flops": 4 * H * case["D"] * _visible(p)}
    if case["op"] == "append":
        return {"bytes": sum(p["rows"]) * 2 * row * (2 + e), "flops": sum(p["rows"]) * 2 * row}
    if case["op"] == "compact":
        moved = sum(sum(1 for j, s in enumerate(w) if s >= 0 and s != j) for w in p["path"])
        return {"bytes": 4 * case["layers"] * moved * row * e + 4 * len(p["lens"]) * 19, "flops": 0}
    kids, ps = case["kids"], case["ps"]
    copies = sum(kids for n in p["lens"] if n % ps)
    blocks = sum(_cdiv(n, ps) for n in p["lens"])
    return {"bytes": 4 * case["layers"] * copies * ps * row * e + 4 * blocks * (1 + 4 * kids), "flops": 0}


# ------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(case, pages, layers, gen, scales):
    shape = (layers, pages, case["ps"], case["G"], case["D"])
    x = torch.randn(shape, dtype=torch.bfloat16, device=DEV, generator=gen)
    if case["kv"] == "bf16":
        return x
    return (x / scales.view(layers, 1, 1, -1, 1).to(torch.bfloat16)).clamp_(-E4M3_MAX, E4M3_MAX).to(
        torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * int(seed) + 17)
    p = _plan(case)
    B, ps, G, D, layers = case["B"], case["ps"], case["G"], case["D"], case.get("layers", 1)
    s = dict(case=case, **{k: _i32(p[k] if p[k] else [0]) for k in ("pos_off", "node_off", "parent", "n_accept")})
    s["kind"], s["path"], s["len"] = _i32(p["kinds"]), _i32(p["path"]), _i32(p["lens"])
    kids = case.get("kids", 0)
    blocks = [_cdiv(n + r, ps) for n, r in zip(p["lens"], p["rows"])]
    if case["op"] == "pages":
        blocks = [_cdiv(n, ps) for n in p["lens"]]
    slots, used = B * (1 + kids), sum(blocks)
    pages = used + max(4, used // 8) + 2 * B * kids
    width = max(blocks) + 2
    # the pages of a cache that has been in use lie in any order
    order = torch.randperm(pages, generator=gen, device=DEV)[:used].to(torch.int32)
    table = torch.full((slots, width), -1, dtype=torch.int32, device=DEV)
    where_b = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(blocks, device=DEV))
    first = torch.tensor([sum(blocks[:b]) for b in range(B)], device=DEV)
    table[where_b, torch.arange(used, device=DEV) - first[where_b]] = order
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[order.long()] = 1
    # a scale for each layer and head of an 8-bit cache: powers of two near amax / 448
    powers = torch.tensor([1 / 128, 1 / 64, 1 / 32], device=DEV)
    sc = [powers[torch.randint(0, 3, (layers, G), generator=gen, device=DEV)] for _ in range(2)]
    s["k_scale"], s["v_scale"] = sc if case["kv"] == "e4m3" else (None, None)
    s.update(table=table, ref=ref, K=_pool(case, pages, layers, gen, sc[0]), V=_pool(case, pages, layers, gen, sc[1]))
    P = p["pos_off"][-1]
    if case["op"] == "attention":
        s["q"] = torch.randn((P, case["H"], D), dtype=torch.bfloat16, device=DEV, generator=gen)
        s["max_rows"] = max(p["rows"])
    if case["op"] == "append":
        # keys and values as one projection leaves them: side by side in a row
        kv = torch.randn((P, 2, G, D), dtype=torch.bfloat16, device=DEV, generator=gen)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    if case["op"] == "pages":
        s["len"] = torch.cat([s["len"], torch.zeros(B * kids, dtype=torch.int32, device=DEV)])
        s["keep"] = s["len"].clone()
        s["src"] = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(kids)
        s["dst"] = torch.arange(B, slots, dtype=torch.int32, device=DEV)
        s["pos_off"] = torch.arange(slots + 1, dtype=torch.int32, device=DEV)   # one new row each
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        s["cache"] = wf.PagedCache(s["K"], s["V"], s["table"], ref=s["ref"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        s["ws"] = wf.PagedWorkspace(slots, H=case.get("H", G), G=G, D=D, max_rows=s.get("max_rows", 1))
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    return {"attention": _attention, "append": _append, "compact": _compact, "pages": _pages}[s["case"]["op"]](s)


def _attention(s):
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        one = s["case"]["form"] == "one"
        out, lse = wf.wf_paged_attention(s["cache"], s["q"], s["pos_off"], s["len"], s["ws"],
                                         node_off=None if one else s["node_off"], kind=None if one else s["kind"],
                                         parent=None if one else s["parent"], max_rows=s["max_rows"], with_lse=True)
        return {"out": out, "lse": lse}
    c = s["case"]
    B, H, G, D, ps, R = c["B"], c["H"], c["G"], c["D"], c["ps"], s["max_rows"]
    hq = H // G
    table, length, pos_off = s["table"], s["len"].long(), s["pos_off"].long()
    T = table.shape[1] * ps
    rows = pos_off[1:] - pos_off[:-1]
    pick = table.clamp(min=0).long()

    def dense(pool, scale):
        x = pool[0][pick].reshape(B, T, G, D).permute(0, 2, 1, 3).float()
        return x if scale is None else x * scale[0].view(1, G, 1, 1)

    r = torch.arange(R, device=DEV)
    t = torch.arange(T, device=DEV)
    live = t[None] < (length + rows)[:, None]                                   # [B, T]
    V = torch.where(live[:, None, :, None], dense(s["V"], s["v_scale"]), 0.0)
    K = dense(s["K"], s["k_scale"])
    at = (pos_off[:-1, None] + r[None]).clamp(max=s["q"].shape[0] - 1)           # [B, R]
    q = s["q"][at].float().reshape(B, R, G, hq, D).permute(0, 2, 1, 3, 4).reshape(B, G, R * hq, D)
    scores = (q @ K.transpose(2, 3) / math.sqrt(D)).reshape(B, G, R, hq, T)
    see = _sees(s, R)                                                           # [B, R, R]
    j = t[None] - length[:, None]                                               # [B, T]
    inside = torch.gather(see, 2, j.clamp(0, R - 1)[:, None].expand(B, R, T))
    mask = (j < 0)[:, None] | (inside & live[:, None])                          # [B, R, T]
    scores = torch.where(mask[:, None, :, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(B, G, R * hq, T) @ V).reshape(B, G, R, hq, D) / total
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, R, H, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, R, H)
    # the packed rows: which (sequence, row) each one is
    p = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(pos_off[1:].contiguous(), p, right=True)
    return {"out": o[b, p - pos_off[b]].to(torch.bfloat16), "lse": lse[b, p - pos_off[b]]}


def _sees(s, R):
    """[B, R, R]: row i of a sequence sees row j (itself, the root and its ancestors; in a chain all before it)."""
    pos_off, node_off = s["pos_off"].long(), s["node_off"].long()
    i = torch.arange(R, device=DEV)
    rows = (pos_off[1:] - pos_off[:-1])[:, None]
    at = (node_off[:-1, None] + i[None] - 1).clamp(0, s["parent"].numel() - 1)
    up = torch.where((i[None] > 0) & (i[None] < rows), 1 + s["parent"].long()[at], 0)     # [B, R] parent row
    step = (i[None, None] == up[:, :, None]) | (i[None, None] == i[None, :, None])
    reach = step.float()
    for _ in range(max(1, (R - 1).bit_length())):                               # ancestors 1, 2, 4, ... above
        reach = (reach @ reach > 0).float()
    return reach > 0


def _append(s):
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        wf.wf_paged_append(s["cache"], s["k"], s["v"], s["pos_off"], s["len"], s["ws"])
    else:
        ps, pos_off = s["case"]["ps"], s["pos_off"].long()
        p = torch.arange(s["k"].shape[0], device=DEV)
        b = torch.searchsorted(pos_off[1:].contiguous(), p, right=True)
        t = s["len"].long()[b] + p - pos_off[b]
        page = s["table"][b, t // ps].long()
        for pool, x, scale in ((s["K"], s["k"], s["k_scale"]), (s["V"], s["v"], s["v_scale"])):
            if scale is not None:
                y = (x.float() / scale[0].view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(pool.dtype)
                pool[0].view(torch.uint8)[page, t % ps] = y.view(torch.uint8)
            else:
                pool[0][page, t % ps] = x
    return {"K": s["K"], "V": s["V"]}


def _compact(s):
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        new_len = wf.wf_paged_compact(s["cache"], s["n_accept"], s["path"], s["len"], s["ws"])
    else:
        ps, path, length = s["case"]["ps"], s["path"].long(), s["len"].long()
        B, S = path.shape
        j = torch.arange(S, device=DEV)[None].expand(B, S)
        kept = j < s["n_accept"][:, None]
        # a column past the path moves the root's row onto itself
        frm = torch.where(kept, length[:, None] + 1 + path, length[:, None])
        to = torch.where(kept, length[:, None] + 1 + j, length[:, None])
        b = torch.arange(B, device=DEV)[:, None].expand(B, S)
        pf, pt = s["table"][b, frm // ps].long(), s["table"][b, to // ps].long()
        for pool in (s["K"], s["V"]):
            raw = pool if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)
            raw[:, pt, to % ps] = raw[:, pf, frm % ps]
        new_len = s["len"] + s["n_accept"] + 1
    return {"K": s["K"], "V": s["V"], "new_len": new_len}


def _pages(s):
    """One step of parallel sampling: last step's continuations go, new ones fork, each gets room for its row."""
    if own:
        from speculative_decoding_verify_lm_gb300 import wf
        wf.wf_pages_trim(s["cache"], s["keep"], s["ws"])
        wf.wf_pages_fork(s["cache"], s["src"], s["dst"], s["len"], s["ws"])
        added = wf.wf_pages_reserve(s["cache"], s["pos_off"], s["len"], s["ws"])
    else:
        ps, table, ref = s["case"]["ps"], s["table"], s["ref"]
        slots, width = table.shape
        col = torch.arange(width, device=DEV)[None]

        def count(entries, chosen, by):
            ref.index_add_(0, torch.where(chosen, entries, 0).reshape(-1).long(),
                           (chosen.to(torch.int32) * by).reshape(-1))

        # trim
        past = (col >= ((s["keep"] + ps - 1) // ps)[:, None]) & (table >= 0)
        count(table, past, -1)
        table[past] = -1
        # fork
        src, dst = s["src"].long(), s["dst"].long()
        length = s["len"][src]
        shared = torch.where(col < ((length + ps - 1) // ps)[:, None], table[src], -1)
        table[dst] = shared
        s["len"][dst] = length
        count(shared, shared >= 0, 1)
        # reserve: one new row each, so one block at most is missing or shared
        length = s["len"].long()
        b = torch.arange(slots, device=DEV)
        blk = length // ps
        page = table[b, blk]
        held = page >= 0
        old = page.clamp(min=0).long()
        # sequences before this one that write into the same page
        before = ((page[None] == page[:, None]) & held[:, None] & (b[None] < b[:, None])).sum(1)
        split = held & (ref[old] - before > 1)
        need = ~held | split
        rank = need.long().cumsum(0) - 1
        spare = ref == 0
        slot_of = torch.where(spare, spare.long().cumsum(0) - 1, ref.numel())
        order = torch.zeros(ref.numel() + 1, dtype=torch.long, device=DEV)
        order[slot_of] = torch.arange(ref.numel(), device=DEV)                  # the free pages, lowest first
        got = order[rank.clamp(min=0)]
        count(page, split, -1)
        count(got, need, 1)
        table[b, blk] = torch.where(need, got.to(torch.int32), page)
        copy = split & (length % ps > 0)
        frm = torch.where(copy, old, table[b, blk].long())                       # else a page onto itself
        to = table[b, blk].long()
        for pool in (s["K"], s["V"]):
            raw = pool if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)
            raw[:, to] = raw[:, frm]
        added = need.to(torch.int32)
    return {"table": s["table"], "ref": s["ref"], "len": s["len"], "added": added, "K": s["K"],
            "V": s["V"]}


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    p, ps = _plan(case), case["ps"]
    if case["op"] == "attention":
        return _exact_attention(case, s, p)
    table = s["table"].tolist()
    pools = {"K": s["K"].double() if case["kv"] == "bf16" else s["K"].float().double(),
             "V": s["V"].double() if case["kv"] == "bf16" else s["V"].float().double()}
    if case["op"] == "append":
        for b in range(case["B"]):
            for i in range(p["rows"][b]):
                t, row = p["lens"][b] + i, p["pos_off"][b] + i
                for name, x, scale in (("K", s["k"], s["k_scale"]), ("V", s["v"], s["v_scale"])):
                    y = x[row].double()
                    if scale is not None:
                        y = _nearest_e4m3(y / scale[0].double()[:, None])
                    pools[name][0, table[b][t // ps], t % ps] = y
        return pools
    if case["op"] == "compact":
        new_len = []
        for b in range(case["B"]):
            n, base = p["n_accept"][b], p["lens"][b] + 1
            for pool in pools.values():
                rows = [pool[:, table[b][(base + p["path"][b][j]) // ps], (base + p["path"][b][j]) % ps].clone()
                        for j in range(n)]
                for j, row in enumerate(rows):
                    pool[:, table[b][(base + j) // ps], (base + j) % ps] = row
            new_len.append(base + n)
        return {**pools, "new_len": _i32(new_len)}
    # pages: sequence after sequence, as the rules are told
    ref, length = s["ref"].tolist(), s["len"].tolist()
    kids, B = case["kids"], case["B"]
    for i in range(B * kids):
        a, b = i // kids, B + i
        length[b] = length[a]
        for j in range(_cdiv(length[a], ps)):
            table[b][j] = table[a][j]
            ref[table[a][j]] += 1
    added = []
    for b in range(len(table)):
        j = length[b] // ps
        old = table[b][j]
        if old >= 0 and ref[old] <= 1:
            added.append(0)
            continue
        new = ref.index(0)
        ref[new], table[b][j] = 1, new
        if old >= 0:
            ref[old] -= 1
            if length[b] % ps:
                for pool in pools.values():
                    pool[:, new] = pool[:, old]
        added.append(1)
    return {"table": _i32(table), "ref": _i32(ref), "len": _i32(length), "added": _i32(added), **pools}


def _nearest_e4m3(x):
    """The nearest value of 8 bits with 4 of exponent and 3 of mantissa, ties to the even one, largest 448."""
    a = x.abs().clamp(max=E4M3_MAX)
    edges = torch.tensor([2.0 ** e for e in range(-6, 9)], dtype=torch.float64, device=x.device)
    step = (edges / 8)[torch.searchsorted(edges, a.contiguous(), right=True).sub(1).clamp(min=0)]
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_attention(case, s, p):
    H, G, D, ps = case["H"], case["G"], case["D"], case["ps"]
    hq = H // G
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, length = p["rows"][b], p["lens"][b]
        T, r0 = length + n, p["pos_off"][b]
        ids = s["table"][b, :_cdiv(T, ps)].long()
        see = torch.zeros(n, T, dtype=torch.bool)
        see[:, :length] = True
        for i in range(n):
            j = i
            while j > 0:
                see[i, length + j] = True
                j = 1 + p["parent"][p["node_off"][b] + j - 1]
            see[i, length] = True
        hide = ~see.to(DEV)
        for g in range(G):
            K, V = ((x[0][ids, :, g].float().double().reshape(-1, D)[:T]) for x in (s["K"], s["V"]))
            if s["k_scale"] is not None:
                K, V = K * s["k_scale"][0, g].double(), V * s["v_scale"][0, g].double()
            q = s["q"][r0:r0 + n, g * hq:(g + 1) * hq].double()
            z = torch.einsum("rhd,td->rht", q, K) / math.sqrt(D)
            z = z.masked_fill(hide[:, None], -math.inf)
            lse[r0:r0 + n, g * hq:(g + 1) * hq] = torch.logsumexp(z, -1)
            out[r0:r0 + n, g * hq:(g + 1) * hq] = torch.softmax(z, -1) @ V
    return {"out": out, "lse": lse}
