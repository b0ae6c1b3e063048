"""The paged cache on the GPU against plain 64-bit references (paged_ref):
attention of single tokens, chains and trees, appended and compacted rows, and
the pages' bookkeeping.  Positions that no sequence owns hold NaN throughout."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import DEV, dev, host
from speculative_decoding_verify_lm_gb300 import wf

pytestmark = pytest.mark.gpu

BAD = 5


def cache_of(c, **kw):
    return wf.PagedCache(c.K.to(DEV), c.V.to(DEV), dev(c.table), k_scale=dev(c.k_scale) if c.kv == "e4m3" else None,
                         v_scale=dev(c.v_scale) if c.kv == "e4m3" else None, **kw)


def run_attention(c, cache=None, scale=None, max_rows=None, q=None, ws=None, trees=None):
    cache = cache or cache_of(c)
    mr = max(max(c.rows), 1) if max_rows is None else max_rows
    ws = ws or wf.PagedWorkspace(c.B, c.H, c.G, c.D, mr)
    trees = any(c.kinds) if trees is None else trees
    out = torch.full((c.P, c.H, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.P, c.H), 7.0, dtype=torch.float32, device=DEV)
    wf.wf_paged_attention(cache, c.q.to(DEV) if q is None else q, dev(c.pos_off), dev(np.array(c.lens, np.int32)), ws,
                          node_off=dev(c.node_off) if trees else None,
                          kind=dev(np.array(c.kinds, np.int32)) if trees else None,
                          parent=dev(c.parent) if trees else None, max_rows=mr, layer=c.layer, scale=scale, out=out,
                          lse=lse)
    torch.cuda.synchronize()
    return host(out.float()).astype(np.float64), host(lse).astype(np.float64), ws


def check(c, scale=None, **kw):
    out, lse, ws = run_attention(c, scale=scale, **kw)
    assert ws.device_error() == (0, 0)
    ro, rl, to, tl = ref.attention(c, c.D ** -0.5 if scale is None else scale)
    mine = ~np.isnan(rl)
    assert np.all(np.abs(out - ro)[mine] <= to[mine]), np.max((np.abs(out - ro) - to)[mine])
    assert np.all(np.abs(lse - rl)[mine] <= tl[mine]), np.max((np.abs(lse - rl) - tl)[mine])
    # rows of no sequence are left as they were
    assert np.all(out[~mine] == 7.0) and np.all(lse[~mine] == 7.0)
    return out, lse


# lens, rows, H, G, D, ps
ONE = [
    ((0,), (1,), 4, 2, 64, 16),                             # the first token: it sees itself alone
    ((1, 62, 63, 64, 65, 127), (1,) * 6, 8, 2, 128, 16),    # around a tile's end
    ((200, 0, 7), (1, 0, 1), 8, 8, 64, 8),                  # a sequence without a row, one head a group
    ((500,), (1,), 32, 8, 80, 16),                          # the drafter's geometry
    ((1000, 3), (1, 1), 20, 1, 96, 32),                     # 20 heads over one: two tiles of pairs
    ((333,), (1,), 4, 4, 16, 8),                            # the smallest head
    ((90, 91), (1, 1), 12, 4, 48, 64),
    ((300,), (1,), 7, 1, 112, 128),
    ((5000,), (1,), 2, 1, 64, 1024),                        # split over many CTAs, one large page size
    (tuple(range(40, 240)), (1,) * 200, 2, 1, 32, 16),      # more sequences than threads
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,H,G,D,ps", ONE)
def test_single_tokens(lens, rows, H, G, D, ps, kv):
    check(ref.Case(1, lens, rows, H, G, D, ps, kv))


# lens, rows, kinds, H, G, D, ps
ROUNDS = [
    ((0,), (2,), (0,), 2, 1, 32, 8),
    ((50,), (17,), (0,), 8, 2, 128, 16),                    # a chain of 16
    ((130,), (61,), (1,), 8, 2, 64, 16),                    # a tree of 60
    ((63, 64, 0, 10), (17, 61, 5, 0), (0, 1, 1, 0), 8, 2, 128, 16),   # mixed, one without a row
    ((300,), (257,), (1,), 2, 1, 16, 32),                   # the largest round
    ((100, 700), (61, 17), (1, 0), 10, 2, 80, 16),          # five heads a group
    ((20, 31), (33, 32), (1, 1), 16, 1, 96, 8),
    ((1500,), (4,), (0,), 4, 2, 112, 64),
    ((9, 8, 7), (3, 2, 1), (1, 1, 1), 1, 1, 128, 8),
    ((129, 255), (128, 129), (0, 1), 3, 1, 48, 16),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,kinds,H,G,D,ps", ROUNDS)
def test_rounds(lens, rows, kinds, H, G, D, ps, kv):
    check(ref.Case(2, lens, rows, H, G, D, ps, kv, kinds=kinds))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,kinds,H,G,D,ps", [
    # a dozen tiles and several pieces a CTA: one product of rows and two, changing within a stretch
    ((2500, 1900, 2222, 700, 2600, 1), (150, 17, 200, 1, 61, 130), (1, 0, 1, 0, 1, 1), 8, 8, 64, 16),
    ((3000,) * 9, (140, 5) * 4 + (129,), (1,) * 9, 8, 8, 32, 64),
    # pieces of one tile next to each other
    (tuple(range(20, 140, 2)), (3,) * 60, (1,) * 60, 8, 8, 16, 8),
])
def test_many_tiles(lens, rows, kinds, H, G, D, ps, kv):
    check(ref.Case(9, lens, rows, H, G, D, ps, kv, kinds=kinds))


def test_many_tiles_of_single_tokens():
    check(ref.Case(10, (9000, 100, 5000, 7000), (1,) * 4, 16, 8, 32, 32))


def test_all_chains_without_a_tree_description():
    c = ref.Case(3, (40, 5), (9, 17), 4, 2, 64, 16)
    check(c, trees=False)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_layers_strided_queries_and_rows_outside(kv):
    """Layer 2 of 3, queries inside a wider projection's rows, rows before the first and behind the last sequence."""
    c = ref.Case(4, (70, 33), (5, 1), 8, 2, 64, 16, kv, kinds=(1, 0), layers=3, layer=2, extra_rows=3, first_row=2)
    wide = torch.randn((c.P, 12, 64), device=DEV).to(torch.bfloat16)
    wide[:, :8] = c.q.to(DEV)
    check(c, q=wide[:, :8])


@pytest.mark.parametrize("scale", [1e-3, 1.0, 8.0])
def test_scales(scale):
    """Nearly uniform weights, and scores far apart (the running maximum moves often)."""
    check(ref.Case(5, (900, 70), (1, 20), 4, 2, 64, 16, kinds=(0, 1), spread=2.0), scale=scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_masked_values_that_are_not_finite(kv):
    """A drafted row whose key and value are not finite reaches only the rows that see it."""
    c = ref.Case(6, (45,), (40,), 8, 2, 64, 16, kv, kinds=(1,))
    c.parent[:] = [-1 if i < 4 else int(c.rng.integers(0, i)) for i in range(39)]
    see = c.sees(0)
    j = 1 + 3                                                # node 3, a child of the root
    t = c.lens[0] + j
    clean_k, clean_v = c.K.clone(), c.V.clone()
    spots = ("V", "K")
    for which in spots:
        c.K, c.V = clean_k.clone(), clean_v.clone()
        pool = c.V if which == "V" else c.K
        bad = float("inf") if kv == "bf16" and which == "V" else float("nan")
        pool[0, c.table[0, t // c.ps], t % c.ps, 1, 5] = bad
        out, lse, ws = run_attention(c)
        assert ws.device_error() == (0, 0)
        c.K, c.V = clean_k, clean_v
        ro, rl, to, tl = ref.attention(c, c.D ** -0.5)
        hit = see[:, j]
        assert hit.any() and not hit.all()
        for i in range(c.rows[0]):
            good = np.abs(out[i] - ro[i]) <= to[i]
            if not hit[i]:
                assert good.all(), (which, i)
            elif which == "V":
                assert good[:4].all() and good[4:, [d for d in range(64) if d != 5]].all()
                assert not np.isfinite(out[i, 4:, 5]).any()
            else:
                assert good[:4].all() and np.isnan(out[i, 4:]).all()


def test_repeated_calls_give_the_same_bits():
    c = ref.Case(7, (3000, 10, 1200), (1, 1, 1), 8, 2, 128, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(3, 8, 2, 128)
    a = run_attention(c, cache, ws=ws)
    for _ in range(3):
        b = run_attention(c, cache, ws=ws)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("what", ["parent", "rows", "length", "page", "long", "nodes"])
def test_bad_sequences_are_nan_and_alone(what):
    c = ref.Case(8, (100, 64, 30), (9, 9, 9), 4, 2, 64, 16, kinds=(1, 1, 1))
    cache = cache_of(c)
    ws = wf.PagedWorkspace(3, 4, 2, 64, 9)
    good = run_attention(c, cache, ws=ws)
    assert ws.device_error() == (0, 0)
    keep_lens, mr = list(c.lens), 9
    if what == "parent":
        c.parent = c.parent.copy()
        c.parent[8 + 4] = 4                                  # its own index
    elif what == "rows":
        mr = 8
    elif what == "length":
        c.lens[1] = -1
    elif what == "long":
        c.lens[1] = c.max_pages * c.ps - 8
    elif what == "page":
        t = c.table.copy()
        t[1, 2] = c.num_pages
        cache = wf.PagedCache(cache.K, cache.V, dev(t))
    elif what == "nodes":
        c.node_off = c.node_off.copy()
        c.node_off[2:] += 1
        c.parent = np.concatenate([c.parent, [0]]).astype(np.int32)
    out, lse, _ = run_attention(c, cache, ws=ws, max_rows=mr)
    code, info = ws.device_error()
    # with the offsets moved by one, the last sequence's parents are its neighbours' and
    # one of them is its own index: whichever of the two is met first is told
    assert code == BAD and info in {"rows": (0, 1, 2), "nodes": (1, 2)}.get(what, (1,))
    hit = slice(0, 27) if what == "rows" else slice(9, 18)
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    if what not in ("rows", "nodes"):
        for s in (slice(0, 9), slice(18, 27)):
            assert np.array_equal(out[s], good[0][s]) and np.array_equal(lse[s], good[1][s])
    elif what == "nodes":
        assert np.array_equal(out[:9], good[0][:9])
    c.lens = keep_lens
    # the workspace is as good as before
    assert ws.device_error() == (0, 0)


def test_identity_table_reads_the_catch_up_cache():
    """The catch-up's cache as a one-layer pool: its attention over the final token, again through the pages."""
    import pins
    case = pins.catchup_case(31, din=256, H=8, G=2, D=64, n=(5, 9), L=(40, 100), cap=128)
    Kc, Vc = dev(case["Kc"]), dev(case["Vc"])
    cu = wf.Catchup(dev(case["u"]), dev(case["bl_off"]), dev(case["cache_len"]), dev(case["gamma"]), dev(case["Wk"]),
                    dev(case["Wv"]), Kc, Vc, 2, Wq=dev(case["Wq"]), Wo=dev(case["Wo"]), eps=case["eps"],
                    theta=case["theta"])
    cu()
    torch.cuda.synchronize()
    B, cap, G, D, H, ps = 2, 128, 2, 64, 8, 16
    c = ref.Case(32, (44, 108), (1, 1), H, G, D, ps)
    c.num_pages, c.max_pages = B * cap // ps, cap // ps
    c.table = np.arange(B * cap // ps, dtype=np.int32).reshape(B, cap // ps)
    c.K = Kc.view(torch.bfloat16).cpu().view(1, -1, ps, G, D)
    c.V = Vc.view(torch.bfloat16).cpu().view(1, -1, ps, G, D)
    check(c)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,G,D,ps", [
    ((0,), (1,), 1, 16, 8),
    ((5, 0, 31, 7), (17, 0, 61, 1), 2, 80, 16),
    ((100,) * 70, (3,) * 70, 4, 64, 32),
    ((15, 16), (1, 257), 8, 128, 8),
])
def test_append(lens, rows, G, D, ps, kv):
    c = ref.Case(11, lens, rows, G, G, D, ps, kv, layers=2, layer=1, extra_rows=2, first_row=1)
    cache = cache_of(c)
    x = torch.randn((c.P, 2, G, D), device=DEV).mul_(40).to(torch.bfloat16)
    if kv == "e4m3":
        x[0, :, 0, 0] = float("inf")
    ws = wf.PagedWorkspace(c.B, G, G, D)
    wf.wf_paged_append(cache, x[:, 0], x[:, 1], dev(c.pos_off), dev(np.array(lens, np.int32)), ws, layer=1)
    torch.cuda.synchronize()
    assert ws.device_error() == (0, 0)
    for i, (pool, was, sc) in enumerate(((cache.K, c.K, c.k_scale), (cache.V, c.V, c.v_scale))):
        want = was.float().numpy().astype(np.float64)
        src = x[:, i].float().cpu().numpy().astype(np.float64)
        for b in range(c.B):
            for r in range(rows[b]):
                t = lens[b] + r
                y = src[c.pos_off[b] + r]
                if sc is not None:
                    # the quotient is a 32-bit number before it is rounded to 8 bits
                    y = (y.astype(np.float32) / sc[1][:, None]).astype(np.float64)
                    y = ref.nearest_e4m3(y)
                want[1, c.table[b, t // ps], t % ps] = y
        got = pool.float().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


def test_append_saturates_and_keeps_nan():
    c = ref.Case(12, (0,), (1,), 1, 1, 16, 8, "e4m3")
    cache = cache_of(c)
    k = torch.zeros((1, 1, 16), dtype=torch.bfloat16, device=DEV)
    k[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30])
    ws = wf.PagedWorkspace(1, 1, 1, 16)
    wf.wf_paged_append(cache, k, k, dev(c.pos_off), dev(np.array([0], np.int32)), ws)
    got = cache.K[0, c.table[0, 0], 0, 0].float().cpu().numpy()
    assert got[0] == 448 and got[1] == -448 and np.isnan(got[2]) and got[3] == 448 and (got[4:] == 0).all()


def test_append_without_a_page():
    c = ref.Case(13, (14, 3), (4, 4), 2, 2, 32, 16)
    t = c.table.copy()
    t[0, 1] = -1                                             # positions 16, 17 of sequence 0
    cache = wf.PagedCache(c.K.to(DEV), c.V.to(DEV), dev(t))
    x = torch.randn((8, 2, 32), device=DEV).to(torch.bfloat16)
    ws = wf.PagedWorkspace(2, 2, 2, 32)
    wf.wf_paged_append(cache, x, x, dev(c.pos_off), dev(np.array([14, 3], np.int32)), ws)
    torch.cuda.synchronize()
    assert ws.device_error() == (BAD, 0)
    want = c.K.clone()
    xc = x.cpu()
    want[0, c.table[0, 0], 14:16] = xc[:2]
    want[0, c.table[1, 0], 3:7] = xc[4:]
    assert torch.equal(torch.nan_to_num(cache.K.cpu()), torch.nan_to_num(want))


# ------------------------------------------------------------------ compact
@pytest.mark.parametrize("kv,in_place", [("bf16", False), ("e4m3", False), ("bf16", True)])
def test_compact(kv, in_place):
    lens, rows = (14, 0, 33, 7, 40, 5), (61, 9, 17, 3, 1, 257)
    c = ref.Case(14, lens, rows, 2, 2, 48, 16, kv, kinds=(1, 1, 0, 1, 1, 1), layers=3)
    S = 40
    path = np.full((6, S), -1, np.int32)
    n = np.array([8, 3, 5, -1, 0, 40], np.int32)
    path[0, :8] = [0, 1, 5, 6, 20, 33, 40, 59]
    path[1, :3] = [2, 3, 7]
    path[2, :5] = range(5)                                   # a chain: nothing moves
    path[5, :40] = np.sort(c.rng.permutation(256)[:40])
    n_call = n.copy()
    n_call[5] = 200                                          # past the columns: taken as the columns
    cache = cache_of(c)
    ws = wf.PagedWorkspace(6, 2, 2, 48)
    ln = dev(np.array(lens, np.int32))
    new = wf.wf_paged_compact(cache, dev(n_call), dev(path), ln, ws, new_len=ln if in_place else None)
    torch.cuda.synchronize()
    assert ws.device_error() == (0, 0)
    assert np.array_equal(host(new), [23, 4, 39, 7, 41, 46])
    for pool, was in ((cache.K, c.K), (cache.V, c.V)):
        raw = torch.int16 if kv == "bf16" else torch.uint8
        want = was.view(raw).clone()
        src = want.clone()
        for b in range(6):
            for j in range(max(n[b], 0)):
                f, t = lens[b] + 1 + path[b, j], lens[b] + 1 + j
                want[:, c.table[b, t // 16], t % 16] = src[:, c.table[b, f // 16], f % 16]
        assert torch.equal(pool.cpu().view(raw), want)


def test_compact_refuses_bad_paths():
    lens, rows = (14, 3, 9, 2), (9, 9, 9, 9)
    c = ref.Case(15, lens, rows, 1, 1, 16, 8, layers=2)
    path = np.array([[0, 2, 2], [1, 0, 3], [-1, 4, 5], [1, 3, 7]], np.int32)
    n = np.array([3, 3, 3, 3], np.int32)
    t = c.table.copy()
    t[3, 1] = -1                                             # position 2 + 1 + 7 = 10 has no page
    cache = wf.PagedCache(c.K.to(DEV), c.V.to(DEV), dev(t))
    ws = wf.PagedWorkspace(4, 1, 1, 16)
    new = wf.wf_paged_compact(cache, dev(n), dev(path), dev(np.array(lens, np.int32)), ws)
    torch.cuda.synchronize()
    assert ws.device_error()[0] == BAD
    assert np.array_equal(host(new), [-1] * 4)
    assert torch.equal(cache.K.cpu().view(torch.int16), c.K.view(torch.int16))


# ------------------------------------------------------------------ pages
def random_pages(rng, B, width, ps, num_pages, share):
    """Sequences with pages of their own, then some that share another's."""
    table = np.full((B, width), -1, np.int32)
    refs = np.zeros(num_pages, np.int32)
    lens = np.zeros(B, np.int32)
    order = list(rng.permutation(num_pages))
    for b in range(B):
        if b and rng.random() < share:
            a = int(rng.integers(0, b))
            lens[b] = lens[a]
            table[b] = table[a]
            refs[table[b][table[b] >= 0]] += 1
            continue
        lens[b] = rng.integers(0, (width - 2) * ps)
        n = min(-(-int(lens[b]) // ps), len(order))
        lens[b] = min(lens[b], n * ps)
        for j in range(n):
            table[b, j] = order.pop()
            refs[table[b, j]] = 1
    return table, refs, lens


def pages_cache(table, refs, ps, layers=2, G=1, D=16):
    n = len(refs)
    K = torch.arange(layers * n * ps * G * D, device=DEV).remainder_(251).view(layers, n, ps, G, D).to(torch.bfloat16)
    V = (K.float() + 0.5).to(torch.bfloat16)
    cache = wf.PagedCache(K, V, dev(table), ref=dev(refs))
    return cache, wf.PagedWorkspace(table.shape[0], G, G, D), K.clone(), V.clone()


@pytest.mark.parametrize("seed,B,width,num_pages,share,most", [
    (1, 1, 4, 8, 0.0, 3),
    (2, 20, 8, 300, 0.5, 40),
    (3, 70, 6, 500, 0.8, 2),
    (4, 40, 8, 220, 0.3, 60),                                # the pages run out
    (5, 1500, 5, 9000, 0.6, 9),                              # more sequences than threads
    (6, 30, 40, 40000, 0.2, 100),                            # free pages in several chunks
    (7, 10, 5, 31, 1.0, 30),
])
def test_reserve(seed, B, width, num_pages, share, most):
    ps = 8
    rng = np.random.default_rng(seed)
    table, refs, lens = random_pages(rng, B, width, ps, num_pages, share)
    if seed == 6:                                            # the first 30,000 pages are held by others
        refs[:30000] += 1
    rows = rng.integers(0, most + 1, B).astype(np.int32)
    rows = np.minimum(rows, width * ps - lens).astype(np.int32)
    cache, ws, K, V = pages_cache(table, refs, ps)
    pos = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    added = wf.wf_pages_reserve(cache, dev(pos), dev(lens), ws)
    torch.cuda.synchronize()
    assert ws.device_error() == (0, 0)
    t2, r2, a2, copies = ref.reserve(table, refs, lens, rows, ps)
    if seed == 4:
        assert (a2 < 0).any() and (a2 > 0).any()
    assert np.array_equal(host(added), a2)
    assert np.array_equal(host(cache.table), t2)
    assert np.array_equal(host(cache.ref), r2)
    for a, b in copies:
        K[:, b], V[:, b] = K[:, a], V[:, a]
    assert torch.equal(cache.K, K) and torch.equal(cache.V, V)


def test_reserve_leaves_bad_sequences():
    ps = 8
    table = np.array([[0, -1, -1], [1, -1, -1], [-1, -1, -1], [99, -1, -1], [2, -1, -1]], np.int32)
    refs = np.zeros(16, np.int32)
    refs[:3] = 1
    lens = np.array([4, -3, 5, 4, 4], np.int32)              # negative; a position without a page; a page id past the pool
    pos = np.array([0, 8, 9, 10, 11, 12], np.int32)
    cache, ws, K, _ = pages_cache(table, refs, ps)
    added = wf.wf_pages_reserve(cache, dev(pos), dev(lens), ws)
    torch.cuda.synchronize()
    code, info = ws.device_error()
    assert code == BAD and info in (1, 2, 3)
    assert np.array_equal(host(added), [1, -1, -1, -1, 0])
    t = table.copy()
    t[0, 1] = 3
    assert np.array_equal(host(cache.table), t)
    assert np.array_equal(host(cache.ref), [1, 1, 1, 1] + [0] * 12) and torch.equal(cache.K, K)


@pytest.mark.parametrize("seed", [1, 2])
def test_fork_and_trim(seed):
    ps, B, width = 8, 12, 6
    rng = np.random.default_rng(seed)
    table, refs, lens = random_pages(rng, 6, width, ps, 60, 0.3)
    table = np.concatenate([table, np.full((6, width), -1, np.int32)])
    lens = np.concatenate([lens, np.zeros(6, np.int32)]).astype(np.int32)
    cache, ws, K, V = pages_cache(table, refs, ps)
    # good forks; then: twice the same destination, an index out of range, a
    # destination in use, a destination that is a source
    src = np.array([0, 0, 3, 1, 1, 2, 4, 12, 5], np.int32)
    dst = np.array([6, 7, 8, 9, 9, 13, 1, 10, 3], np.int32)
    ln = dev(lens)
    wf.wf_pages_fork(cache, dev(src), dev(dst), ln, ws)
    torch.cuda.synchronize()
    t2, r2, l2, bad = ref.fork(table, refs, lens, src, dst, ps)
    assert bad == [3, 4, 5, 6, 7, 8]
    code, info = ws.device_error()
    assert code == BAD and info in bad
    assert np.array_equal(host(cache.table), t2) and np.array_equal(host(cache.ref), r2)
    assert np.array_equal(host(ln), l2)
    keep = l2.copy()
    keep[[0, 7]] = 0
    keep[3] = keep[3] // 2
    keep[4] = -1                                             # left as it is
    wf.wf_pages_trim(cache, dev(keep), ws)
    torch.cuda.synchronize()
    assert ws.device_error() == (BAD, 4)
    t3, r3 = ref.trim(t2, r2, keep, ps)
    assert np.array_equal(host(cache.table), t3) and np.array_equal(host(cache.ref), r3)
    wf.wf_pages_trim(cache, dev(np.zeros(B, np.int32)), ws)  # everything back
    torch.cuda.synchronize()
    assert (host(cache.ref) == 0).all() and (host(cache.table) == -1).all()
    assert torch.equal(cache.K, K) and torch.equal(cache.V, V)


def test_trim_of_malformed_entries():
    table = np.array([[0, 1, 77, -5], [2, 3, -1, -1]], np.int32)
    refs = np.array([1, 0, 1, 1, 0], np.int32)               # page 1 is held by nobody
    cache, ws, _, _ = pages_cache(table, refs, 8)
    wf.wf_pages_trim(cache, dev(np.array([0, 8], np.int32)), ws)
    torch.cuda.synchronize()
    assert ws.device_error() == (BAD, 0)
    assert np.array_equal(host(cache.table), [[-1] * 4, [2, -1, -1, -1]])
    assert np.array_equal(host(cache.ref), [0, 0, 1, 0, 0])


# ------------------------------------------------------------------ how a program uses them
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,H,G,D", [
    ((70, 300), (5, 9), 20, 1, 96),        # 20 heads a group: six query rows a product
    ((40,), (3,), 128, 1, 16),             # 128: one
    ((200, 10), (1, 1), 16, 2, 64),        # single tokens through the kernel of drafted rows
])
def test_wide_groups_and_single_rows_among_rounds(lens, rows, H, G, D, kv):
    check(ref.Case(41, lens, rows, H, G, D, 16, kv), max_rows=max(rows) + 2)


def test_no_rows_at_all():
    c = ref.Case(42, (5, 6), (0, 0), 4, 2, 32, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(2, 4, 2, 32, 5)
    for mr in (1, 5):
        out, lse = wf.wf_paged_attention(cache, torch.empty((0, 4, 32), dtype=torch.bfloat16, device=DEV),
                                         dev(np.zeros(3, np.int32)), dev(np.array([5, 6], np.int32)), ws, max_rows=mr,
                                         with_lse=True)
        assert out.shape == (0, 4, 32) and lse.shape == (0, 4)
        q = torch.zeros((3, 4, 32), dtype=torch.bfloat16, device=DEV)   # rows that no sequence has
        out = torch.full((3, 4, 32), 7.0, dtype=torch.bfloat16, device=DEV)
        wf.wf_paged_attention(cache, q, dev(np.zeros(3, np.int32)), dev(np.array([5, 6], np.int32)), ws, max_rows=mr,
                              out=out)
        torch.cuda.synchronize()
        assert (out == 7.0).all() and ws.device_error() == (0, 0)


@pytest.mark.parametrize("rows", [1, 9])
def test_pools_past_32_bit_offsets(rows):
    """Pages whose elements lie past 2^31 (and bytes past 2^32), with the rest of the pool never written."""
    H, G, D, ps, num = 8, 8, 128, 64, 33100          # 33,100 x 64 x 1,024 elements
    c = ref.Case(43, (150,), (rows,), H, G, D, ps)
    used = [int(p) for p in c.table[0] if p >= 0]
    K = torch.empty((1, num, ps, G, D), dtype=torch.bfloat16, device=DEV)
    V = torch.empty_like(K)
    table = c.table.copy()
    for i, p in enumerate(used):
        table[0, i] = num - 1 - i
        K[0, num - 1 - i], V[0, num - 1 - i] = c.K[0, p].to(DEV), c.V[0, p].to(DEV)
    cache = wf.PagedCache(K, V, dev(table))
    check(c, cache=cache)
    ws = wf.PagedWorkspace(1, H, G, D)
    x = torch.randn((rows, G, D), device=DEV).to(torch.bfloat16)
    wf.wf_paged_append(cache, x, x, dev(c.pos_off), dev(np.array([150], np.int32)), ws)
    torch.cuda.synchronize()
    t = 150 + rows - 1
    assert torch.equal(K[0, table[0, t // ps], t % ps], x[-1]) and ws.device_error() == (0, 0)


def test_captured_and_replayed_with_new_lengths():
    """One graph of append, attention and compaction; the lengths and pages change between its replays."""
    c = ref.Case(44, (90, 20), (9, 9), 8, 2, 64, 16, kinds=(1, 1), slack=8)
    cache = cache_of(c)
    ws = wf.PagedWorkspace(2, 8, 2, 64, 9)
    q, pos, node = c.q.to(DEV), dev(c.pos_off), dev(c.node_off)
    par, kind = dev(c.parent), dev(np.ones(2, np.int32))
    ln = dev(np.array(c.lens, np.int32))
    kv = torch.randn((18, 2, 2, 64), device=DEV).to(torch.bfloat16)
    n_acc = dev(np.array([2, 1], np.int32))
    path = dev(np.array([[0, 4, -1], [3, -1, -1]], np.int32))
    new = torch.zeros(2, dtype=torch.int32, device=DEV)

    def step():
        wf.wf_paged_append(cache, kv[:, 0], kv[:, 1], pos, ln, ws)
        out, lse = wf.wf_paged_attention(cache, q, pos, ln, ws, node_off=node, kind=kind, parent=par, max_rows=9,
                                         with_lse=True)
        wf.wf_paged_compact(cache, n_acc, path, ln, ws, new_len=new)
        return out, lse

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step()
    for lens in ((90, 20), (3, 23), (60, 0)):   # within the two sequences' pages
        K0, V0 = cache.K.clone(), cache.V.clone()
        ln.copy_(dev(np.array(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        assert ws.device_error() == (0, 0)
        assert np.array_equal(host(new), [lens[0] + 3, lens[1] + 2])
        c.lens = list(lens)
        c.K, c.V = K0.cpu(), V0.cpu()
        for b in range(2):
            for r in range(9):
                pg, at = c.table[b, (lens[b] + r) // 16], (lens[b] + r) % 16
                c.K[0, pg, at], c.V[0, pg, at] = kv[9 * b + r, 0].cpu(), kv[9 * b + r, 1].cpu()
        ro, rl, to, tl = ref.attention(c, 0.125)
        assert np.all(np.abs(host(out.float()).astype(np.float64) - ro) <= to)
        assert np.all(np.abs(host(lse).astype(np.float64) - rl) <= tl)


def test_two_streams_with_a_workspace_each():
    cs = [ref.Case(45 + i, (2000 - 700 * i, 300), (1, 1) if i else (20, 17), 8, 2, 64, 16, kinds=(1, 0) if not i else None)
          for i in range(2)]
    caches = [cache_of(c) for c in cs]
    want = [run_attention(c, k) for c, k in zip(cs, caches)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [wf.PagedWorkspace(2, 8, 2, 64, 20) for _ in range(2)]
    args = [(c.q.to(DEV), dev(c.pos_off), dev(np.array(c.lens, np.int32)), dev(c.node_off),
             dev(np.array(c.kinds, np.int32)), dev(c.parent)) for c in cs]
    outs = [[torch.empty((c.P, 8, 64), dtype=torch.bfloat16, device=DEV) for _ in range(6)] for c in cs]
    torch.cuda.synchronize()
    for r in range(6):
        for i in range(2):
            q, pos, ln, node, kind, par = args[i]
            wf.wf_paged_attention(caches[i], q, pos, ln, wss[i], node_off=None if i else node, kind=None if i else kind,
                                  parent=None if i else par, max_rows=1 if i else 20, out=outs[i][r], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert wss[i].device_error() == (0, 0)
        for o in outs[i]:
            assert np.array_equal(host(o.float()).astype(np.float64), want[i][0])


def test_rounds_of_speculation_over_a_paged_cache():
    """Reserve, append, attend, verify, compact, trim over several rounds of forked sequences, against lists of rows."""
    rng = np.random.default_rng(50)
    H, G, D, ps, B, layers, R = 4, 2, 32, 8, 4, 2, 13
    num, width = 40, 12
    K = torch.full((layers, num, ps, G, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    V = K.clone()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(num, dtype=torch.int32, device=DEV)
    cache = wf.PagedCache(K, V, table, ref=refs)
    ws = wf.PagedWorkspace(B, H, G, D, R)
    vws = wf.Workspace(B * R, B)
    ln = torch.zeros(B, dtype=torch.int32, device=DEV)
    rows_of = [[] for _ in range(B)]                         # per sequence: (layers' keys, layers' values) of its positions

    def append(rows, kv):
        pos = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        added = wf.wf_pages_reserve(cache, dev(pos), ln, ws)
        for layer in range(layers):
            wf.wf_paged_append(cache, kv[:, layer, 0], kv[:, layer, 1], dev(pos), ln, ws, layer=layer)
        assert (host(added) >= 0).all()
        return pos

    def new_rows(n):
        return torch.from_numpy(rng.standard_normal((n, layers, 2, G, D))).to(torch.bfloat16).to(DEV)

    # two prompts, each forked once
    rows = [11, 0, 16, 0]
    kv = new_rows(sum(rows))
    pos = append(rows, kv)
    for b in range(B):
        rows_of[b] = [kv[pos[b] + i] for i in range(rows[b])]
    ln += dev(np.array(rows, np.int32))
    wf.wf_pages_fork(cache, dev(np.array([0, 2], np.int32)), dev(np.array([1, 3], np.int32)), ln, ws)
    rows_of[1], rows_of[3] = list(rows_of[0]), list(rows_of[2])
    assert host(ln).tolist() == [11, 11, 16, 16]
    for step in range(4):
        rows = [R, 1, 7, R] if step % 2 else [5, R, R, 2]
        kinds = np.array([1, 0, 1, 1], np.int32)
        P = sum(rows)
        kv, q = new_rows(P), torch.from_numpy(rng.standard_normal((P, H, D))).to(torch.bfloat16).to(DEV)
        node = np.concatenate([[0], np.cumsum([r - 1 for r in rows])]).astype(np.int32)
        par = np.array([int(rng.integers(max(-1, i - 4), i)) if kinds[b] else i - 1
                        for b in range(B) for i in range(rows[b] - 1)] or [0], np.int32)
        tok = rng.integers(0, 2, len(par)).astype(np.int32)  # two tokens: paths are accepted a few deep
        target = rng.integers(0, 2, P).astype(np.int32)
        pos = append(rows, kv)
        before = host(ln).copy()
        for layer in range(layers):
            out, lse = wf.wf_paged_attention(cache, q, dev(pos), ln, ws, node_off=dev(node), kind=dev(kinds),
                                             parent=dev(par), max_rows=R, layer=layer, with_lse=True)
            # the same through the plain reference on the rows as the lists have them
            c = ref.Case.__new__(ref.Case)
            c.H, c.G, c.D, c.ps, c.kv, c.layer, c.B = H, G, D, ps, "bf16", 0, B
            c.lens, c.rows, c.kinds, c.P = [int(x) for x in before], rows, list(kinds), P
            c.q, c.pos_off, c.node_off, c.parent = q.cpu(), pos, node, par
            c.k_scale = c.v_scale = None
            c.dense = lambda b, g, which: torch.stack(  # noqa: E731
                [r[layer, 0 if which == "K" else 1, g] for r in rows_of[b]] +
                [kv[pos[b] + i, layer, 0 if which == "K" else 1, g] for i in range(rows[b])]).float().cpu().numpy().astype(np.float64)
            ro, rl, to, tl = ref.attention(c, D ** -0.5)
            assert np.all(np.abs(host(out.float()) - ro) <= to) and np.all(np.abs(host(lse) - rl) <= tl)
        S = R - 1
        # chains and trees as one verification of trees: a chain's parents are its predecessors
        n_t, _, _, path_t = wf.wf_verify_tree(dev(target), dev(tok), dev(par), dev(node), dev(pos), vws, path_stride=S)
        new = wf.wf_paged_compact(cache, n_t, path_t, ln, ws, new_len=ln)
        assert new is ln
        n_acc, path = host(n_t), host(path_t)
        wf.wf_pages_trim(cache, ln, ws)
        torch.cuda.synchronize()
        assert ws.device_error() == (0, 0) and vws.device_error() == (0, 0)
        for b in range(B):
            rows_of[b].append(kv[pos[b]])
            rows_of[b] += [kv[pos[b] + 1 + int(path[b, j])] for j in range(int(n_acc[b]))]
            assert int(ln[b]) == len(rows_of[b]) == before[b] + n_acc[b] + 1
        # every position of every sequence is the row it should be, in every layer
        t = host(table)
        for b in range(B):
            for i, r in enumerate(rows_of[b]):
                for layer in range(layers):
                    assert torch.equal(K[layer, t[b, i // ps], i % ps], r[layer, 0])
                    assert torch.equal(V[layer, t[b, i // ps], i % ps], r[layer, 1])
            assert (t[b, -(-len(rows_of[b]) // ps):] == -1).all()
        count = np.zeros(num, np.int32)
        for p in t[t >= 0]:
            count[p] += 1
        assert np.array_equal(host(refs), count)
    wf.wf_pages_trim(cache, torch.zeros_like(ln), ws)
    assert (host(refs) == 0).all()


def test_binding_refuses_wrong_tensors():
    c = ref.Case(51, (20, 20), (3, 3), 4, 2, 32, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(2, 4, 2, 32, 3)
    pos, ln, q = dev(c.pos_off), dev(np.array(c.lens, np.int32)), c.q.to(DEV)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :16]), dict(q=q.transpose(0, 1)), dict(pos_off=pos[:2]),
                dict(cache_len=ln.long()), dict(cache_len=ln.cpu()), dict(out=torch.empty(3, device=DEV))):
        kw = dict(q=q, pos_off=pos, cache_len=ln, out=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            wf.wf_paged_attention(cache, kw["q"], kw["pos_off"], kw["cache_len"], ws, max_rows=3, out=kw["out"])
    with pytest.raises(wf.WfError):
        wf.wf_paged_attention(cache, q, pos, ln, ws, max_rows=3, layer=1)
    with pytest.raises(wf.WfError):
        wf.wf_pages_trim(cache, ln, ws)                      # no reference counts
    with pytest.raises(ValueError):
        wf.PagedCache(cache.K, cache.V[:, :1], cache.table)
    with pytest.raises(ValueError):
        wf.PagedCache(cache.K, cache.V, cache.table, k_scale=torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        wf.PagedWorkspace(2, 5, 2, 32)
    small = wf.PagedWorkspace(2, 4, 2, 32, 1)                # made for single tokens
    with pytest.raises(wf.WfError):
        wf.wf_paged_attention(cache, q, pos, ln, small, max_rows=3)


def test_a_sequence_of_several_rows_among_single_tokens_is_nan():
    c = ref.Case(60, (70, 9, 200), (1, 1, 1), 20, 2, 64, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(3, 20, 2, 64)
    good = run_attention(c, cache, ws=ws)
    c.pos_off = np.array([0, 1, 4, 5], np.int32)             # the second sequence has three rows
    c.P = 6
    c.q = torch.cat([c.q[:1], c.q[1:2].expand(3, -1, -1), c.q[2:], c.q[:1]]).contiguous()
    out, lse, _ = run_attention(c, cache, ws=ws, max_rows=1)
    assert ws.device_error() == (BAD, 1)
    assert np.isnan(out[1:4]).all() and np.isnan(lse[1:4]).all()
    for new, old in ((0, 0), (4, 2)):
        assert np.array_equal(out[new], good[0][old]) and np.array_equal(lse[new], good[1][old])
    assert (out[5] == 7.0).all() and (lse[5] == 7.0).all()


@pytest.mark.parametrize("rows", [1, 3])
def test_keys_of_minus_infinity_weigh_nothing(rows):
    """Scores of -inf, over whole tiles and whole warps' shares of one, are weights of 0 and no NaN."""
    c = ref.Case(61, (700,), (rows,), 4, 2, 64, 16)
    c.q[:, :, 0] = c.q[:, :, 0].abs() + 0.125
    outs = []
    for low in (float("-inf"), -2.0 ** 100):
        K = c.K.clone()
        for t in [*range(0, 300), *range(320, 336), *range(400, 464), 500]:
            c.K[0, c.table[0, t // 16], t % 16, :, 0] = low
        outs.append(run_attention(c))
        c.K = K
    assert np.isfinite(outs[0][0]).all() and np.isfinite(outs[0][1]).all()
    assert np.array_equal(outs[0][0], outs[1][0]) and np.array_equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("rows", [1, 3])
def test_keys_that_are_nan_make_the_rows_nan(rows):
    c = ref.Case(62, (700,), (rows,), 4, 2, 64, 16)
    for t in range(320, 336):
        c.K[0, c.table[0, t // 16], t % 16, 1, 3] = float("nan")
    out, lse, ws = run_attention(c)
    assert ws.device_error() == (0, 0)
    assert np.isfinite(out[:, :2]).all() and np.isfinite(lse[:, :2]).all()
    assert np.isnan(out[:, 2:]).all() and np.isnan(lse[:, 2:]).all()


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("power", [-120, 120])
def test_queries_of_any_size_over_an_8_bit_cache(rows, power):
    """Queries times 2^n against keys over 2^n: the same bits."""
    c = ref.Case(63, (300,), (rows,), 8, 2, 64, 16, "e4m3")
    c.q[0, 0] = 0                                            # a head without a direction: it weighs all alike
    c.q = (c.q.float() * 2.0 ** power).to(torch.bfloat16)    # the least elements become subnormal and round
    far_q = c.q.clone()
    c.q = (far_q.double() * 2.0 ** -power).to(torch.bfloat16)   # exact: what the call far out is given
    plain = run_attention(c)
    c.q = far_q
    c.k_scale = (np.asarray(c.k_scale) * 2.0 ** -power).astype(np.float32)
    far = run_attention(c)
    assert np.isfinite(far[0]).all()
    assert np.array_equal(plain[0], far[0]) and np.array_equal(plain[1], far[1])


def test_calls_of_other_shapes_share_a_workspace():
    """A round's reserved pages for a few sequences, then a compaction of many, in one workspace."""
    B, ps = 1500, 8
    ws = wf.PagedWorkspace(B, 1, 1, 16)
    K = torch.zeros((1, 8 * B, ps, 1, 16), dtype=torch.bfloat16, device=DEV)
    few, pages = 600, 7
    refs = torch.zeros(8 * B, dtype=torch.int32, device=DEV)
    small = wf.PagedCache(K, K.clone(), torch.full((few, pages), -1, dtype=torch.int32, device=DEV), refs)
    pos = torch.arange(few + 1, dtype=torch.int32, device=DEV) * (ps * pages)
    added = wf.wf_pages_reserve(small, pos, torch.zeros(few, dtype=torch.int32, device=DEV), ws)
    assert (added == pages).all().item()
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    big = wf.PagedCache(K, K.clone(), table.contiguous())
    ln = torch.full((B,), 3, dtype=torch.int32, device=DEV)
    n_acc = torch.arange(B, dtype=torch.int32, device=DEV) % 3
    path = torch.arange(2, dtype=torch.int32, device=DEV).repeat(B, 1)
    for _ in range(2):
        new = torch.full((B,), -7, dtype=torch.int32, device=DEV)
        wf.wf_paged_compact(big, n_acc, path, ln, ws, new_len=new)
        assert torch.equal(new, ln + n_acc + 1)
    assert ws.device_error() == (0, 0)


def test_host_memory_is_refused():
    """What the kernels copy with the tensor-memory accelerator must be this GPU's memory."""
    c = ref.Case(64, (20, 20), (3, 1), 4, 2, 32, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(2, 4, 2, 32, 3)
    out = torch.full((c.P, 4, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    pos, ln, q = dev(c.pos_off), dev(np.array(c.lens, np.int32)), c.q.to(DEV)
    a = wf.PagedAttnArgs(q=q.data_ptr(), q_stride=4 * 32, P=c.P, H=4, pos_off=pos.data_ptr(), cache_len=ln.data_ptr(),
                         max_rows=3, layer=0, scale=0.25, out=out.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    call = lambda cc, aa: wf.lib().wf_paged_attention(ctypes.byref(cc), ctypes.byref(aa), ws.ptr,  # noqa: E731
                                                      ws.nbytes, stream)
    pinned = torch.zeros(cache.K.numel() * 2, dtype=torch.uint8).pin_memory()
    pageable = torch.zeros(cache.K.numel() * 2 + 64, dtype=torch.uint8)
    for ptr in (pinned.data_ptr(), pageable.data_ptr() + (-pageable.data_ptr()) % 16):
        for field in ("K", "V"):
            other = wf.PagedCacheArgs.from_buffer_copy(cache.args)
            setattr(other, field, ptr)
            assert call(other, a) == 1, field
        other = wf.PagedAttnArgs.from_buffer_copy(a)
        other.q = ptr
        assert call(cache.args, other) == 1
    torch.cuda.synchronize()
    assert (out == 7.0).all().item() and ws.device_error() == (0, 0)
    assert call(cache.args, a) == 0
    torch.cuda.synchronize()
    assert ws.device_error() == (0, 0) and not (out == 7.0).all().item()


def test_workspaces_of_other_calls_are_refused():
    c = ref.Case(65, (20,), (1,), 4, 2, 32, 16)
    with pytest.raises(ValueError):
        wf.wf_paged_attention(cache_of(c), c.q.to(DEV), dev(c.pos_off), dev(np.array(c.lens, np.int32)),
                              wf.Workspace(4096, 4))


@pytest.mark.parametrize("rows", [1, 3])
def test_keys_of_the_lowest_value_weigh_alike(rows):
    """Every score the same, -3.4e38 / 64: the mean of the values, to its sums' and the output's rounding."""
    c = ref.Case(66, (333,), (rows,), 4, 2, 64, 16)
    low = torch.finfo(torch.bfloat16).min
    c.K[:] = 0
    c.K[..., 0] = low
    c.q[:, :, 0] = 0.125
    out, lse, ws = run_attention(c)
    assert ws.device_error() == (0, 0)
    for i in range(rows):
        n = 333 + i + 1
        for h in range(4):
            v = c.dense(0, h // 2, "V")[:n]
            tol = n * 2.0 ** -23 * np.abs(v).mean(0)
            assert np.all(np.abs(out[i, h] - v.mean(0)) <= tol + 2.0 ** -8 * (np.abs(v.mean(0)) + tol))
            assert abs(lse[i, h] - (low * 0.015625 + np.log(n))) <= 2.0 ** -22 * abs(low * 0.015625)


def test_more_sequences_than_threads_in_a_round():
    """1,500 short sequences of one to three rows, some without any."""
    rows = tuple((1, 2, 3, 0, 2)[b % 5] for b in range(1500))
    lens = tuple(7 * b % 90 for b in range(1500))
    check(ref.Case(67, lens, rows, 2, 1, 16, 8, kinds=tuple(b % 2 for b in range(1500))))


@pytest.mark.parametrize("how", ["compact", "in place", "fork", "attention"])
def test_catch_up_right_behind_a_call_that_writes_its_inputs(how):
    """Compaction (into a fresh tensor and in place), forking and attention, each followed at once by a catch-up that
    reads what they write: the bits of a run that waits in between."""
    import pins
    B, cap, G, D, H, ps, layers = 2, 512, 2, 64, 4, 16, 48
    c = pins.catchup_case(70, din=H * D, H=H, G=G, D=D, n=(5, 9), L=(203, 402), cap=cap)
    pages = B * cap // ps
    g = torch.Generator(device=DEV).manual_seed(70)
    K0 = torch.randn((layers, pages, ps, G, D), device=DEV, generator=g).to(torch.bfloat16)
    V0 = torch.randn((layers, pages, ps, G, D), device=DEV, generator=g).to(torch.bfloat16)
    K, V = K0.clone(), V0.clone()
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(B, -1)   # the catch-up's [B, cap, G * D] view
    if how == "fork":    # its lengths come from two sequences that the tables of this cache describe
        table = torch.cat([table, torch.full_like(table, -1)])
    ws = wf.PagedWorkspace(4, H, G, D, 9)
    cache = wf.PagedCache(K, V, table, ref=torch.ones(pages, dtype=torch.int32, device=DEV))
    before = {"fork": [203, 402, 0, 0]}.get(how, [200, 400])
    ln = dev(np.array(before, np.int32))
    lengths = ln if how in ("in place", "fork") else torch.empty_like(ln)
    u = dev(c["u"])
    cu = wf.Catchup(u, dev(c["bl_off"]), lengths[2:] if how == "fork" else lengths, dev(c["gamma"]), dev(c["Wk"]),
                    dev(c["Wv"]), K[1].view(torch.int16).view(B, cap, G * D), V[1].view(torch.int16).view(B, cap, G * D),
                    G, Wq=dev(c["Wq"]), Wo=dev(c["Wo"]), eps=c["eps"], theta=c["theta"])
    n_acc, path = dev(np.array([2, 1], np.int32)), dev(np.array([[3, 5, -1], [4, -1, -1]], np.int32))
    q = torch.randn((14, H, D), device=DEV, generator=g).to(torch.bfloat16)
    pos = dev(np.array([0, 5, 14], np.int32))
    copies, refs = cache.table.clone(), cache.ref.clone()

    def reset():
        K.copy_(K0), V.copy_(V0), ln.copy_(dev(np.array(before, np.int32)))
        cache.table.copy_(copies), cache.ref.copy_(refs), u.copy_(dev(c["u"]))
        if lengths is not ln:
            lengths.fill_(-7 if how == "compact" else 203)

    def first():
        if how == "fork":
            wf.wf_pages_fork(cache, dev_src, dev_dst, ln, ws)
        elif how == "attention":
            wf.wf_paged_attention(cache, q, pos, ln, ws, max_rows=9, layer=2, out=u.view(torch.bfloat16).view(14, H, D))
        else:
            wf.wf_paged_compact(cache, n_acc, path, ln, ws, new_len=lengths)

    dev_src, dev_dst = dev(np.array([0, 1], np.int32)), dev(np.array([2, 3], np.int32))
    seen = []
    for wait in (True, False, False, False):
        reset()
        torch.cuda.synchronize()
        first()
        if wait:
            torch.cuda.synchronize()
        out, attn = cu()
        torch.cuda.synchronize()
        assert ws.device_error() == (0, 0) and cu.ws.device_error() == (0, 0)
        seen.append([x.clone() for x in (out, attn, K, V, lengths)])
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first()
        cu()
    for _ in range(5):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert ws.device_error() == (0, 0) and cu.ws.device_error() == (0, 0)
        seen.append([x.clone() for x in (cu.out, cu.attn, K, V, lengths)])
    assert host(seen[0][4]).tolist() == {"fork": [203, 402, 203, 402], "attention": [203, 203]}.get(how, [203, 402])
    for got in seen[1:]:
        for a, b in zip(got, seen[0]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("block", [2, 6])                    # cached positions; the round's own
def test_any_table_entry_that_is_no_page_is_told(kv, rows, block):
    c = ref.Case(71, (100, 64, 30), (rows,) * 3, 4, 2, 64, 16, kv, kinds=(1, 1, 1))
    cache, ws = cache_of(c), wf.PagedWorkspace(3, 4, 2, 64, 9)
    good = run_attention(c, cache, ws=ws)
    assert ws.device_error() == (0, 0) and np.isfinite(good[0]).all()
    for entry in (-1, -2, -3, -2 ** 31, c.num_pages, 2 ** 31 - 1):
        t = c.table.copy()
        t[0, block] = entry
        other = wf.PagedCache(cache.K, cache.V, dev(t), k_scale=cache.k_scale, v_scale=cache.v_scale)
        out, lse, _ = run_attention(c, other, ws=ws)
        assert ws.device_error() == (BAD, 0), entry
        assert np.isnan(out[:rows]).all() and np.isnan(lse[:rows]).all(), entry
        assert np.array_equal(out[rows:], good[0][rows:]) and np.array_equal(lse[rows:], good[1][rows:])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D", [(10, 2, 80), (12, 1, 64), (8, 2, 128)])
def test_rows_do_not_depend_on_the_product_s_other_rows(kv, H, G, D):
    """The same bits whatever the neighbour's queries are and whatever ran before: rows that are no query of the
    sequence share its products and its warps."""
    c = ref.Case(72, (900, 700), (3, 3), H, G, D, 16, kv)
    cache, ws = cache_of(c), wf.PagedWorkspace(2, H, G, D, 3)
    want = run_attention(c, cache, ws=ws)
    q = c.q.clone()
    # queries that fill every row of the products of another call, each as far out as it gets
    full = ref.Case(73, (300,) * 8, (128,) * 8, 2, 2, D, 16, kv)
    full_cache, full_ws = cache_of(full), wf.PagedWorkspace(8, 2, 2, D, 128)
    for power, what in ((0, 1.0), (60, 1.0), (-60, 1.0), (0, float("nan")), (0, float("inf")), (0, 0.0)):
        fill = torch.randn((8 * 128, 2, D), device=DEV).mul_(what).mul_(2.0 ** power).to(torch.bfloat16)
        c.q = q.clone()
        c.q[3:] = (q[3:].float() * what * 2.0 ** power).to(torch.bfloat16)
        for _ in range(2):
            run_attention(full, full_cache, ws=full_ws, q=fill)
            got = run_attention(c, cache, ws=ws)
            assert np.array_equal(got[0][:3], want[0][:3]) and np.array_equal(got[1][:3], want[1][:3]), (power, what)
    assert ws.device_error() == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_repeated_rounds_give_the_same_bits(kv):
    """Five heads a group (three rows of each product belong to nobody), pieces that are joined, other work between."""
    c = ref.Case(74, (3000, 10, 1200, 2000), (61, 5, 130, 17), 10, 2, 64, 16, kv, kinds=(1, 1, 1, 0))
    cache, ws = cache_of(c), wf.PagedWorkspace(4, 10, 2, 64, 130)
    other = ref.Case(75, (400,) * 40, (40,) * 40, 8, 8, 64, 16, kv)
    other_cache, other_ws = cache_of(other), wf.PagedWorkspace(40, 8, 8, 64, 40)
    a = run_attention(c, cache, ws=ws)
    for i in range(4):
        fill = torch.randn((1600, 8, 64), device=DEV).mul_(float("nan") if i == 3 else 2.0 ** (20 * i)).to(torch.bfloat16)
        run_attention(other, other_cache, ws=other_ws, q=fill)
        b = run_attention(c, cache, ws=ws)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_refuses_a_first_row_without_a_page(in_place):
    """Nothing accepted, or a path that lies in the next page: the first row's own page has to be there."""
    lens, rows = (16, 15, 7, 16), (2, 9, 2, 1)
    c = ref.Case(76, lens, rows, 1, 1, 16, 8, layers=2)
    t = c.table.copy()
    t[0, 2] = -1                                             # position 16, nothing accepted
    t[1, 1] = c.num_pages                                    # position 15, a path that stays in pages 2 and 3
    path = np.array([[-1, -1], [1, 3], [0, -1], [-1, -1]], np.int32)
    n = np.array([0, 2, 1, -1], np.int32)                    # the last keeps no row: its page does not matter
    t[3, 2] = -1
    cache = wf.PagedCache(c.K.to(DEV), c.V.to(DEV), dev(t))
    ws = wf.PagedWorkspace(4, 1, 1, 16)
    ln = dev(np.array(lens, np.int32))
    new = wf.wf_paged_compact(cache, dev(n), dev(path), ln, ws, new_len=ln if in_place else None)
    torch.cuda.synchronize()
    code, info = ws.device_error()
    assert code == BAD and info in (0, 1)
    assert np.array_equal(host(new), [-1, -1, 9, 16])
    assert torch.equal(cache.K.cpu().view(torch.int16), c.K.view(torch.int16))


@pytest.mark.parametrize("H,G,D,n", [(8, 2, 128, 700), (4, 4, 64, 90), (32, 2, 80, 3000), (12, 1, 128, 500)])
def test_single_tokens_weigh_values_to_more_than_16_bits(H, G, D, n):
    """Weights over a bf16 cache: 2^-14 of each off (a product of 2^-8 by the 2^-7 + 2^-9 that the first of its two
    numbers leaves), beside the scores' and sums' fp32 and the output's one rounding."""
    c = ref.Case(77, (n,), (1,), H, G, D, 16)
    out, lse = check(c)
    scale, hq = D ** -0.5, H // G
    for h in range(H):
        K, V, x = c.dense(0, h // hq, "K"), c.dense(0, h // hq, "V"), c.q[0, h].double().numpy()
        s = scale * (K @ x)
        w = np.exp(s - s.max())
        w /= w.sum()
        ds = scale * D * ref.FP32 * (np.abs(K) @ np.abs(x)).max() + 2.0 ** -22 * np.abs(s).max()
        rel = 2.0 ** -14 + 2 * ds + 2.0 ** -20 + 2 * (n + 1) * ref.FP32
        o, mass = w @ V, w @ np.abs(V)
        assert np.all(np.abs(out[0, h] - o) <= rel * mass + ref.BF16 * (np.abs(o) + rel * mass)), h


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_infinite_values_that_a_single_token_sees(kv):
    """An infinite value is the output's infinity in its dim, at any weight above zero, and in no other dim."""
    c = ref.Case(78, (400, 30), (1, 1), 8, 2, 64, 16, kv)
    clean = ref.attention(c, 0.125)
    K = c.dense(0, 1, "K")
    s = K @ c.q[0, 4].double().numpy()
    for t in (int(s.argmax()), int(s.argmin()), 0, 400):     # the largest weight (1 before the sum), the least, the ends
        V = c.V.clone()
        spot = V[0, c.table[0, t // 16], t % 16, 1]
        spot[3], spot[9] = (float("inf"), float("-inf")) if kv == "bf16" else (float("nan"),) * 2
        was, c.V = c.V, V
        out, lse, ws = run_attention(c)
        c.V = was
        assert ws.device_error() == (0, 0)
        hit = np.zeros(out.shape, bool)
        hit[0, 4:, [3, 9]] = True
        assert np.all(np.abs(out - clean[0])[~hit] <= clean[2][~hit])
        assert np.all(np.abs(lse - clean[1]) <= clean[3])
        if kv == "bf16":
            assert (out[0, 4:, 3] == np.inf).all() and (out[0, 4:, 9] == -np.inf).all()
        else:
            assert np.isnan(out[hit]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_shared_pages_are_not_written(kv):
    """A reserve that finds no page leaves a sequence on shared pages; the round's append and compaction leave those
    pages to the others, whose rows they hold."""
    ps, G, D = 8, 1, 16
    c = ref.Case(79, (13, 20), (6, 2), G, G, D, ps, kv, layers=2)
    table = np.full((2, 5), -1, np.int32)
    table[0, :2], table[1, :3] = [4, 1], [4, 1, 2]           # two pages in common; the first is shorter by 7 rows
    refs = np.array([1, 2, 1, 1, 2], np.int32)               # none is free
    cache = wf.PagedCache(c.K[:, :5].contiguous().to(DEV), c.V[:, :5].contiguous().to(DEV), dev(table), ref=dev(refs),
                          k_scale=dev(c.k_scale) if kv == "e4m3" else None,
                          v_scale=dev(c.v_scale) if kv == "e4m3" else None)
    was = [x.clone().view(torch.uint8) for x in (cache.K, cache.V)]
    ws = wf.PagedWorkspace(2, G, G, D)
    pos, ln = dev(np.array([0, 3, 5], np.int32)), dev(np.array([13, 20], np.int32))
    added = wf.wf_pages_reserve(cache, pos, ln, ws)
    assert host(added).tolist() == [-1, -1] and ws.device_error() == (0, 0)
    x = torch.randn((5, G, D), device=DEV).to(torch.bfloat16)
    wf.wf_paged_append(cache, x, x, pos, ln, ws, layer=1)
    torch.cuda.synchronize()
    assert ws.device_error() == (BAD, 0)
    # the first sequence's rows are dropped, the second's are in its own page
    t1 = [int(table[1, t // ps]) * ps + t % ps for t in (20, 21)]
    for pool, w in ((cache.K, was[0]), (cache.V, was[1])):
        left = torch.ones(5 * ps, dtype=torch.bool)
        left[t1] = False
        got, want = pool.view(torch.uint8).view(2, 5 * ps, -1).cpu(), w.view(2, 5 * ps, -1).cpu()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1][left], want[1][left])
        assert not torch.equal(got[1][t1], want[1][t1])
    was = [x_.clone().view(torch.uint8) for x_ in (cache.K, cache.V)]
    n, path = dev(np.array([1, 1], np.int32)), dev(np.array([[1, -1], [0, -1]], np.int32))
    new = wf.wf_paged_compact(cache, n, path, ln, ws)
    assert host(new).tolist() == [-1, 22] and ws.device_error() == (BAD, 0)
    for pool, w in zip((cache.K, cache.V), was):
        assert torch.equal(pool.view(torch.uint8), w)


@pytest.mark.parametrize("first", [-1, -5, -2 ** 31 + 40, -2 ** 31])
def test_append_behind_a_negative_first_row(first):
    """Offsets that no batch has: the rows are dropped and told of, at whatever distance from the first."""
    c = ref.Case(80, (30, 9), (4, 4), 2, 2, 32, 16)
    cache, ws = cache_of(c), wf.PagedWorkspace(2, 2, 2, 32)
    x = torch.randn((8, 2, 32), device=DEV).to(torch.bfloat16)
    wf.wf_paged_append(cache, x, x, dev(np.array([first, 4, 8], np.int64).astype(np.int32)),
                       dev(np.array(c.lens, np.int32)), ws)
    torch.cuda.synchronize()
    assert ws.device_error() == (BAD, 0)
    want = c.K.clone()
    want[0, c.table[1, 0], 9:13] = x[4:].cpu()
    assert torch.equal(cache.K.cpu().view(torch.int16), want.view(torch.int16))
