"""The heads' log-probabilities and the draft head's distillation refuse bad arguments on the host, before any device
is touched, and the references the GPU tests compare with agree with hand-worked cases."""
import ctypes
import math

import pytest
import torch

import heads_ref as ref
from speculative_decoding_verify_lm_gb300 import wf

INVALID, WORKSPACE = 1, 2
BIG = 1 << 40


def logprobs(ws=256, nbytes=BIG, **kw):
    a = wf.LogprobsArgs()
    a.hidden = a.W = a.tok = a.logp = a.lse = a.H = a.top_ids = a.top_logp = 256
    a.P, a.d, a.V, a.S, a.k, a.temperature = 5, 64, 100, 2, 4, 1.0
    for n, v in kw.items():
        setattr(a, n, v)
    return wf.lib().wf_lmhead_logprobs(ctypes.byref(a), ws, nbytes, None)


def distill(fn, ws=256, nbytes=BIG, **kw):
    a = wf.DistillArgs()
    a.x = a.Wd = a.tid = a.tlogit = a.t2d = a.z = a.lse = a.loss = a.gloss = a.dx = a.dWd = 256
    a.N, a.d, a.Vd, a.k, a.V, a.temperature, a.ldz = 5, 64, 100, 4, 300, 1.0, 100
    for n, v in kw.items():
        setattr(a, n, v)
    return getattr(wf.lib(), fn)(ctypes.byref(a), ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(hidden=None), dict(W=None), dict(hidden=264), dict(W=258), dict(P=0), dict(P=-1), dict(d=60), dict(d=0),
    dict(d=16392), dict(V=0), dict(V=2 ** 31 - 1), dict(S=0), dict(S=65), dict(S=-1), dict(tok=None), dict(logp=None),
    dict(k=17), dict(k=-1), dict(k=4, V=3), dict(top_ids=None, top_logp=None), dict(temperature=0.0),
    dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf), dict(temperature=1e-40),
    dict(temperature=2.5e-39), dict(tok=None, S=0, k=0, lse=None, H=None),
])
def test_logprobs_arguments_are_checked(kw):
    assert logprobs(**kw) == INVALID


@pytest.mark.parametrize("fn", ["wf_draft_distill", "wf_draft_distill_grad"])
@pytest.mark.parametrize("kw", [
    dict(x=None), dict(Wd=None), dict(x=264), dict(Wd=258), dict(N=0), dict(d=60), dict(Vd=0), dict(Vd=2 ** 31 - 1),
    dict(tid=None), dict(tlogit=None), dict(lse=None), dict(k=0), dict(k=65), dict(V=0), dict(t2d=None),
    dict(temperature=0.0), dict(temperature=math.nan), dict(temperature=1e-45), dict(z=264), dict(ldz=99),
    dict(ldz=102), dict(ldz=(1 << 34) + 4), dict(ldz=96),
])
def test_distill_arguments_are_checked(fn, kw):
    assert distill(fn, **kw) == INVALID


@pytest.mark.parametrize("fn,kw", [
    ("wf_draft_distill", dict(loss=None)), ("wf_draft_distill_grad", dict(z=None)),
    ("wf_draft_distill_grad", dict(dx=None, dWd=None)), ("wf_draft_distill_grad", dict(dx=264)),
    ("wf_draft_distill_grad", dict(dWd=258)),
    ("wf_draft_distill_grad", dict(N=2 ** 30, Vd=10 ** 8, ldz=10 ** 8)),     # more tiles than an int counts
])
def test_each_distill_call_checks_its_own(fn, kw):
    assert distill(fn, **kw) == INVALID


def test_workspaces_are_checked():
    L = wf.lib()
    n = L.wf_logprobs_workspace_bytes(5, 64, 100, 2, 4)
    m = L.wf_distill_workspace_bytes(5, 64, 100, 4)
    assert n > 256 and m > 256 and n % 256 == m % 256 == 0
    for ws, size in ((None, BIG), (256 + 64, BIG), (256, n - 1)):
        assert logprobs(ws, size) == WORKSPACE
    for fn in ("wf_draft_distill", "wf_draft_distill_grad"):
        for ws, size in ((None, BIG), (256 + 64, BIG), (256, m - 1)):
            assert distill(fn, ws, size) == WORKSPACE


def test_workspace_sizes():
    L = wf.lib()
    size = L.wf_logprobs_workspace_bytes
    assert [size(0, 64, 100, 1, 1), size(5, 60, 100, 1, 1), size(5, 64, 3, 1, 4), size(5, 64, 100, 65, 1),
            size(5, 64, 100, 1, 17), size(5, 64, 100, -1, 1)] == [0] * 6
    # a state of 144 bytes a row and pair of CTAs; bounded where a call takes its rows in chunks
    assert size(4096, 2560, 151936, 1, 16) >= 4096 * 76 * 144
    assert size(1 << 20, 2560, 151936, 1, 16) < size(4096, 2560, 151936, 1, 16) * 8
    size = L.wf_distill_workspace_bytes
    assert [size(0, 64, 100, 4), size(5, 64, 0, 4), size(5, 64, 100, 0), size(5, 64, 100, 65)] == [0] * 4
    assert 2 * 4096 * 32000 <= size(4096, 2560, 32000, 10) <= 4 * 4096 * 32000
    # a workspace for the most rows serves fewer
    for N in (1, 64, 127, 128, 129, 300, 777, 4096, 20000):
        assert size(N, 2560, 32000, 10) <= size(N + 1, 2560, 32000, 10)
        assert L.wf_logprobs_workspace_bytes(N, 2560, 32000, 1, 10) <= L.wf_logprobs_workspace_bytes(
            N + 1, 2560, 32000, 1, 10)


def test_ids_that_an_int_does_not_count_in_steps():
    """Draft vocabularies from 2^30 on: the pass over a row's logits would step past 2^31."""
    for fn in ("wf_draft_distill", "wf_draft_distill_grad"):
        assert distill(fn, Vd=2 ** 30, ldz=2 ** 30) == INVALID
    size = wf.lib().wf_distill_workspace_bytes
    assert size(1, 8, 2 ** 30, 1) == 0 and size(1, 8, 2 ** 30 - 1, 1) >= 2 ** 31


def test_the_binding_refuses_before_the_library():
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        wf.wf_lmhead_logprobs(x, W, None)
    with pytest.raises(ValueError, match="CUDA"):
        wf.wf_draft_distill(x, W, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), None)
    with pytest.raises(ValueError, match="z is required"):
        wf.wf_draft_distill_grad(x, W, None, None, None, None, None)
    with pytest.raises(ValueError, match="neither"):
        wf.wf_draft_distill_grad(x, W, None, None, x, None, None, need_dx=False, need_dWd=False)


# ------------------------------------------------------------------ the references by hand
def test_logprobs_by_hand():
    """Logits (0, log 2, log 4): probabilities 1/7, 2/7, 4/7."""
    x = torch.tensor([[1.0, 0, 0, 0, 0, 0, 0, 0]])
    W = torch.zeros(3, 8)
    W[1, 0], W[2, 0] = math.log(2), math.log(4)
    r, _ = ref.logprobs(x, W, 1.0, torch.tensor([[1, -1, 2]]), 2)
    assert torch.allclose(r["lse"], torch.tensor([math.log(7)], dtype=torch.float64))
    assert torch.allclose(r["logp"], torch.tensor([[math.log(2 / 7), 0, math.log(4 / 7)]], dtype=torch.float64))
    h = -(math.log(1 / 7) + 2 * math.log(2 / 7) + 4 * math.log(4 / 7)) / 7
    assert abs(float(r["H"][0]) - h) < 1e-7 and r["top_ids"].tolist() == [[2, 1]]
    # at temperature 2 the odds are the square roots: 1 : sqrt 2 : 2
    r, _ = ref.logprobs(x, W, 2.0, torch.tensor([0]), 0)
    assert abs(float(r["logp"][0]) + math.log(3 + math.sqrt(2))) < 1e-7


def test_distill_by_hand():
    """Student odds 1 : 2 : 4; a teacher with equal odds on ids 0 and 2 (one through the map, one place empty)."""
    x = torch.tensor([[1.0, 0, 0, 0, 0, 0, 0, 0], [0.0] * 8])
    W = torch.zeros(3, 8)
    W[1, 0], W[2, 0] = math.log(2), math.log(4)
    t2d = torch.tensor([2, -1, 0, 1], dtype=torch.int32)
    tid = torch.tensor([[0, 1, 2, -1], [1, -1, -1, -1]], dtype=torch.int32)
    r = ref.distill(x, W, tid, torch.tensor([[3.0, 9.0, 3.0, math.nan], [0.0] * 4]), t2d, 1.0)
    assert r["some"].tolist() == [True, False]
    assert abs(float(r["loss"][0]) - (math.log(.5) - .5 * math.log(4 / 7) - .5 * math.log(1 / 7))) < 1e-7
    assert float(r["loss"][1]) == 0
    dx, dW, _, _ = ref.grads(x, W, r, None, 1.0)
    G = [1 / 7 - .5, 2 / 7, 4 / 7 - .5]
    assert abs(float(dx[0, 0]) - (G[1] * math.log(2) + G[2] * math.log(4))) < 1e-7 and not bool(dx[1].any())
    assert torch.allclose(dW[:, 0], torch.tensor(G, dtype=torch.float64), atol=1e-7) and not bool(dW[:, 1:].any())


def test_packed_arguments_are_the_structures_bytes():
    """The binding packs what include/wf.h lays out: every field at its place."""
    import struct
    for fmt, cls in ((wf._LOGPROBS, wf.LogprobsArgs), (wf._DISTILL, wf.DistillArgs)):
        values = [float(i + 2) if t is ctypes.c_float else i + 2 for i, (_, t) in enumerate(cls._fields_)]
        a = cls(*values)
        assert fmt.size == ctypes.sizeof(cls) and isinstance(fmt, struct.Struct)
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert [getattr(got, n) for n, _ in cls._fields_] == [getattr(a, n) for n, _ in cls._fields_] == values
