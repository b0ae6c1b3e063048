"""The paged cache's calls refuse bad arguments on the host, before any device
is touched, and the references the GPU tests compare with agree with hand-worked
cases."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from speculative_decoding_verify_lm_gb300 import wf

INVALID, WORKSPACE = 1, 2


def cache(**kw):
    a = wf.PagedCacheArgs()
    a.K = a.V = a.table = a.ref = 256
    a.kv_type, a.layers, a.num_pages, a.page_size, a.G, a.D, a.B, a.max_pages = 0, 2, 10, 16, 2, 64, 3, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attn(**kw):
    a = wf.PagedAttnArgs()
    a.q = a.pos_off = a.cache_len = a.out = 256
    a.q_stride, a.P, a.H, a.max_rows, a.layer, a.scale = 8 * 64, 5, 8, 17, 0, 0.125
    for k, v in kw.items():
        setattr(a, k, v)
    return a


WS = (256, 1 << 30)


def calls(c, a=None):
    L, p = wf.lib(), ctypes.byref(c)
    a = a or attn()
    return {
        "append": L.wf_paged_append(p, 0, 256, c.G * c.D, 256, c.G * c.D, 5, 256, 256, *WS, None),
        "attention": L.wf_paged_attention(p, ctypes.byref(a), *WS, None),
        "compact": L.wf_paged_compact(p, 256, 256, 4, 256, 256, *WS, None),
        "reserve": L.wf_pages_reserve(p, 256, 256, 256, *WS, None),
        "fork": L.wf_pages_fork(p, 256, 256, 1, 256, *WS, None),
        "trim": L.wf_pages_trim(p, 256, *WS, None),
    }


@pytest.mark.parametrize("kw", [
    dict(K=None), dict(V=264), dict(table=None), dict(kv_type=2), dict(layers=0), dict(num_pages=0),
    dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(G=0), dict(D=72), dict(D=144), dict(B=0),
    dict(B=4097), dict(max_pages=0), dict(num_pages=1 << 27), dict(max_pages=(1 << 26) + 1), dict(k_scale=256),
    dict(G=129, D=128), dict(layers=1 << 26),
])
def test_cache_descriptions_are_checked(kw):
    got = calls(cache(**kw))
    assert set(got.values()) == {INVALID}, got


def test_pages_need_reference_counts():
    got = calls(cache(ref=None))
    assert all(got[k] == INVALID for k in ("reserve", "fork", "trim"))
    if not torch.cuda.is_available():   # (a device then refuses these addresses, which are none of its memory's)
        assert all(got[k] != INVALID for k in ("append", "attention", "compact"))


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=264), dict(out=None), dict(out=264), dict(pos_off=None), dict(cache_len=None),
    dict(parent=256), dict(q_stride=504), dict(q_stride=516), dict(P=-1), dict(H=7), dict(H=1), dict(max_rows=0),
    dict(max_rows=258), dict(layer=2), dict(layer=-1), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=-1.0),
])
def test_attention_arguments_are_checked(kw):
    assert wf.lib().wf_paged_attention(ctypes.byref(cache()), ctypes.byref(attn(**kw)), *WS, None) == INVALID


def test_other_arguments_are_checked():
    L, c = wf.lib(), ctypes.byref(cache())
    ap = lambda **k: L.wf_paged_append(c, k.get("layer", 0), k.get("k", 256), k.get("ks", 128), k.get("v", 256),  # noqa: E731
                                       k.get("vs", 128), k.get("P", 5), k.get("pos", 256), k.get("len", 256), *WS, None)
    for k in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=264), dict(ks=120), dict(vs=132), dict(P=-1),
              dict(pos=None), dict(len=None)):
        assert ap(**k) == INVALID, k
    assert L.wf_paged_compact(c, None, 256, 4, 256, 256, *WS, None) == INVALID
    assert L.wf_paged_compact(c, 256, None, 4, 256, 256, *WS, None) == INVALID
    assert L.wf_paged_compact(c, 256, 256, -1, 256, 256, *WS, None) == INVALID
    assert L.wf_paged_compact(c, 256, 256, 257, 256, 256, *WS, None) == INVALID
    assert L.wf_paged_compact(c, 256, 256, 4, 256, None, *WS, None) == INVALID
    assert L.wf_pages_reserve(c, None, 256, None, *WS, None) == INVALID
    assert L.wf_pages_fork(c, 256, 256, -1, 256, *WS, None) == INVALID
    assert L.wf_pages_fork(c, 256, 256, 4, 256, *WS, None) == INVALID       # more forks than sequences
    assert L.wf_pages_fork(c, 256, 256, 1, None, *WS, None) == INVALID
    assert L.wf_pages_trim(c, None, *WS, None) == INVALID
    assert L.wf_pages_trim(None, 256, *WS, None) == INVALID


def test_workspace():
    L = wf.lib()
    n = L.wf_paged_workspace_bytes(3, 8, 2, 64, 17)
    assert n > 0 and n % 256 == 0
    for bad in ((0, 8, 2, 64, 17), (4097, 8, 2, 64, 17), (3, 7, 2, 64, 17), (3, 258, 2, 64, 17), (3, 8, 2, 60, 17),
                (3, 8, 2, 64, 0), (3, 8, 2, 64, 258)):
        assert L.wf_paged_workspace_bytes(*bad) == 0, bad
    c, a = ctypes.byref(cache()), ctypes.byref(attn())
    for ws in ((None, n), (256 + 64, n), (256, n - 256)):
        assert L.wf_paged_attention(c, a, *ws, None) == WORKSPACE
        assert L.wf_pages_trim(c, 256, ws[0], 256, None) == WORKSPACE


def test_reference_reserve_by_hand():
    # page 0 is shared by two sequences of 4 positions (pages of 8); page 1 is one's own
    table = np.array([[0, -1], [0, -1], [1, -1]], np.int32)
    t, r, added, copies = ref.reserve(table, np.array([2, 1, 0, 0, 0], np.int32), [4, 4, 8], [1, 1, 1], 8)
    assert t.tolist() == [[2, -1], [0, -1], [1, 3]]           # the last holder keeps the shared page
    assert r.tolist() == [1, 1, 1, 1, 0] and added.tolist() == [1, 0, 1] and copies == [(0, 2)]
    t, r, added, copies = ref.reserve(table, np.array([2, 1, 0], np.int32), [4, 4, 8], [1, 1, 1], 8)
    assert t.tolist() == [[2, -1], [0, -1], [1, -1]] and added.tolist() == [1, 0, -1]


def test_reference_e4m3_by_hand():
    x = np.array([0.0, 448.0, 1000.0, -17.0, -18.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 0.0146484375, 1.0625, 1.1875])
    assert ref.nearest_e4m3(x).tolist() == [0.0, 448.0, 448.0, -16.0, -18.0, 2.0 ** -9, 0.0, 2.0 ** -8, 0.015625,
                                            1.0, 1.25]


@pytest.mark.parametrize("scale,refused", [(2.3e38, False), (2.4e38, True), (3.4e38, True), (1e-38, False)])
def test_scales_that_are_infinite_to_base_2_are_refused(scale, refused):
    """The kernels' exponents are scores times scale times log2(e)."""
    got = wf.lib().wf_paged_attention(ctypes.byref(cache()), ctypes.byref(attn(scale=scale)), 256, 256, None)
    assert got == (INVALID if refused else WORKSPACE)
