"""Python binding of ``libwf.so`` (the C ABI declared in include/wf.h).

Argument marshalling only: every function takes torch CUDA tensors, checks
dtype / device / contiguity, and passes raw device pointers and the current
(or given) CUDA stream to the library; all arithmetic runs in the library's
kernels.  The functions carry the C names.  If the shared library is missing
it is built with nvcc; if that fails, loading raises - there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

WF_MAX_SEQ_NODES = 256
WF_MAX_TOPK = 16
WF_KV_BF16, WF_KV_E4M3 = 0, 1
WF_PAGED_MAX_SEQS = 4096
WF_MAX_LISTED = 64
STATUS = {0: "WF_OK", 1: "WF_ERR_INVALID_ARG", 2: "WF_ERR_WORKSPACE", 3: "WF_ERR_CUDA", 4: "WF_ERR_UNSUPPORTED",
          5: "WF_ERR_BAD_DATA", 6: "WF_ERR_TIMEOUT"}


class WfError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().wf_status_string(status).decode()} (status {status})")


_c_void_p = ctypes.c_void_p
_i32 = ctypes.c_int
_f32 = ctypes.c_float
_u64 = ctypes.c_uint64
_sz = ctypes.c_size_t


class RoundArgs(ctypes.Structure):
    """Mirror of ``wf_round_args``."""
    _fields_ = [
        ("hidden", _c_void_p), ("W", _c_void_p), ("P", _i32), ("d", _i32), ("V", _i32),
        ("B", _i32), ("pos_off", _c_void_p), ("node_off", _c_void_p), ("kind", _c_void_p), ("tok", _c_void_p),
        ("parent", _c_void_p), ("path_stride", _i32),
        ("m", _i32), ("W1", _c_void_p), ("b1", _c_void_p), ("w2", _c_void_p), ("b2", _f32), ("tau", _f32),
        ("x", _c_void_p), ("Wd", _c_void_p), ("d2t", _c_void_p), ("Vd", _i32), ("k", _i32),
        ("ids", _c_void_p), ("maxlogit", _c_void_p), ("n_accept", _c_void_p), ("bonus", _c_void_p),
        ("last_pos", _c_void_p), ("path", _c_void_p), ("delta_al", _c_void_p), ("route", _c_void_p),
        ("draft_ids", _c_void_p), ("tids", _c_void_p), ("vals", _c_void_p), ("router_kind", _i32),
        ("lse", _c_void_p),
    ]


WF_ROUTER_NEURAL = 0
WF_ROUTER_ENTROPY = 1


class CatchupArgs(ctypes.Structure):
    """Mirror of ``wf_catchup_args``."""
    _fields_ = [
        ("u", _c_void_p), ("bl_off", _c_void_p), ("cache_len", _c_void_p), ("B", _i32), ("N", _i32), ("din", _i32),
        ("H", _i32), ("G", _i32), ("D", _i32), ("gamma", _c_void_p), ("eps", _f32), ("theta", _f32),
        ("Wq", _c_void_p), ("Wk", _c_void_p), ("Wv", _c_void_p), ("Wo", _c_void_p), ("Kc", _c_void_p),
        ("Vc", _c_void_p), ("cap", _i32), ("out", _c_void_p), ("attn", _c_void_p),
    ]


class PagedCacheArgs(ctypes.Structure):
    """Mirror of ``wf_paged_cache``."""
    _fields_ = [
        ("K", _c_void_p), ("V", _c_void_p), ("k_scale", _c_void_p), ("v_scale", _c_void_p), ("table", _c_void_p),
        ("ref", _c_void_p), ("kv_type", _i32), ("layers", _i32), ("num_pages", _i32), ("page_size", _i32),
        ("G", _i32), ("D", _i32), ("B", _i32), ("max_pages", _i32),
    ]


class PagedAttnArgs(ctypes.Structure):
    """Mirror of ``wf_paged_attn_args``."""
    _fields_ = [
        ("q", _c_void_p), ("q_stride", ctypes.c_int64), ("P", _i32), ("H", _i32), ("pos_off", _c_void_p),
        ("cache_len", _c_void_p), ("node_off", _c_void_p), ("kind", _c_void_p), ("parent", _c_void_p),
        ("max_rows", _i32), ("layer", _i32), ("scale", _f32), ("out", _c_void_p), ("lse", _c_void_p),
    ]


class LogprobsArgs(ctypes.Structure):
    """Mirror of ``wf_logprobs_args``."""
    _fields_ = [
        ("hidden", _c_void_p), ("W", _c_void_p), ("P", _i32), ("d", _i32), ("V", _i32), ("temperature", _f32),
        ("tok", _c_void_p), ("S", _i32), ("k", _i32), ("logp", _c_void_p), ("lse", _c_void_p), ("H", _c_void_p),
        ("top_ids", _c_void_p), ("top_logp", _c_void_p),
    ]


class DistillArgs(ctypes.Structure):
    """Mirror of ``wf_distill_args``."""
    _fields_ = [
        ("x", _c_void_p), ("Wd", _c_void_p), ("N", _i32), ("d", _i32), ("Vd", _i32), ("tid", _c_void_p),
        ("tlogit", _c_void_p), ("k", _i32), ("t2d", _c_void_p), ("V", _i32), ("temperature", _f32), ("z", _c_void_p),
        ("ldz", ctypes.c_int64), ("lse", _c_void_p), ("loss", _c_void_p), ("gloss", _c_void_p), ("dx", _c_void_p),
        ("dWd", _c_void_p),
    ]


# the same bytes as PagedAttnArgs
_PAGED_ATTN = struct.Struct("@PqiiPPPPPiifPP")
# ... as LogprobsArgs and as DistillArgs
_LOGPROBS = struct.Struct("@PPiiifPiiPPPPP")
_DISTILL = struct.Struct("@PPiiiPPiPifPqPPPPP")

_SIGS = {
    "wf_status_string": (ctypes.c_char_p, [_i32]),
    "wf_version": (_i32, []),
    "wf_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "wf_lmhead_entropy": (_i32, [_c_void_p, _i32, _i32, _c_void_p, _i32, _c_void_p, _i32, _f32, _c_void_p, _c_void_p,
                                 _c_void_p, _sz, _c_void_p]),
    "wf_workspace_init": (_i32, [_c_void_p, _sz, _c_void_p]),
    "wf_read_device_error": (_i32, [_c_void_p, ctypes.POINTER(_i32), ctypes.POINTER(_i32), _i32, _c_void_p]),
    "wf_set_wait_timeout_ns": (None, [_u64]),
    "wf_probe_bounded_wait": (_i32, [_u64, _c_void_p, _sz, _c_void_p]),
    "wf_lmhead_argmax": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _sz,
                                _c_void_p]),
    "wf_lmhead_argmax_noalloc": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "wf_noalloc_read_device_error": (_i32, [ctypes.POINTER(_i32), ctypes.POINTER(_i32), _i32, _c_void_p]),
    "wf_build_tree": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                             _c_void_p, _sz, _c_void_p]),
    "wf_accepted_rows": (_i32, [_c_void_p, _c_void_p, _i32, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32,
                                _c_void_p, _c_void_p]),
    "wf_verify_chain": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p,
                               _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_verify_tree": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i32, _c_void_p,
                              _c_void_p, _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_router_mlp": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _f32, _f32,
                             _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_draft_topk": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p,
                             _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_lmhead_draft_topk": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_round": (_i32, [ctypes.POINTER(RoundArgs), _c_void_p, _sz, _c_void_p]),
    "wf_catchup_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "wf_catchup_kv": (_i32, [ctypes.POINTER(CatchupArgs), _c_void_p, _sz, _c_void_p]),
    "wf_catchup": (_i32, [ctypes.POINTER(CatchupArgs), _c_void_p, _sz, _c_void_p]),
    "wf_paged_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "wf_paged_append": (_i32, [ctypes.POINTER(PagedCacheArgs), _i32, _c_void_p, ctypes.c_int64, _c_void_p,
                               ctypes.c_int64, _i32, _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_paged_attention": (_i32, [ctypes.POINTER(PagedCacheArgs), _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_paged_compact": (_i32, [ctypes.POINTER(PagedCacheArgs), _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p,
                                _c_void_p, _sz, _c_void_p]),
    "wf_pages_reserve": (_i32, [ctypes.POINTER(PagedCacheArgs), _c_void_p, _c_void_p, _c_void_p, _c_void_p, _sz,
                                _c_void_p]),
    "wf_pages_fork": (_i32, [ctypes.POINTER(PagedCacheArgs), _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p, _sz,
                             _c_void_p]),
    "wf_pages_trim": (_i32, [ctypes.POINTER(PagedCacheArgs), _c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_logprobs_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "wf_lmhead_logprobs": (_i32, [_c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_distill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "wf_draft_distill": (_i32, [_c_void_p, _c_void_p, _sz, _c_void_p]),
    "wf_draft_distill_grad": (_i32, [_c_void_p, _c_void_p, _sz, _c_void_p]),
}


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load (building first if missing or stale) the native library."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def exported_symbols() -> list:
    return list(_SIGS)


# ------------------------------------------------------------------ marshalling
def _check(t: Optional[torch.Tensor], name: str, dtypes, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.numel() == 0:   # an empty array still needs a valid (never read) device address
        return _placeholder(t.device)
    return t.data_ptr()


_placeholders = {}


def _placeholder(device) -> int:
    if device not in _placeholders:
        _placeholders[device] = torch.zeros(16, dtype=torch.int32, device=device)
    return _placeholders[device].data_ptr()


_BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = torch.cuda.current_device


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(_device())   # torch.cuda.current_stream().cuda_stream, without building the object
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _raise(st: int, where: str):
    if st != 0:
        raise WfError(st, where)


class Workspace:
    """Caller-owned device workspace sized by wf_workspace_bytes and zeroed once."""

    def __init__(self, P: int, B: int = 1, m: int = 1, Vd: int = 0, k: int = 0, device=None, stream=None,
                 d: int = 0):
        self.nbytes = int(lib().wf_workspace_bytes(P, B, d, m, Vd, k))
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        _raise(lib().wf_workspace_init(self.buf.data_ptr(), self.nbytes, _stream(stream)), "wf_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def device_error(self, clear: bool = True, stream=None):
        code, info = _i32(0), _i32(0)
        _raise(lib().wf_read_device_error(self.ptr, ctypes.byref(code), ctypes.byref(info), int(clear),
                                          _stream(stream)), "wf_read_device_error")
        return code.value, info.value


def wf_workspace_bytes(P: int, B: int = 1, m: int = 1, Vd: int = 0, k: int = 0, d: int = 0) -> int:
    return int(lib().wf_workspace_bytes(P, B, d, m, Vd, k))


def wf_lmhead_entropy(hidden, W, tau: float, ws: Workspace, rows=None, B=None, H=None, route=None, stream=None):
    """Entropy of the target's next-token distribution at the given rows (all rows if None) and the
    WhiFlash-Entropy route (H > tau)."""
    P, d = hidden.shape
    V = W.shape[0]
    B = (rows.numel() if rows is not None else P) if B is None else B
    H = torch.empty(B, dtype=torch.float32, device=hidden.device) if H is None else H
    route = torch.empty(B, dtype=torch.int32, device=hidden.device) if route is None else route
    st = lib().wf_lmhead_entropy(_check(hidden, "hidden", _BF16), P, d, _check(rows, "rows", _I32, True), B,
                                 _check(W, "W", _BF16), V, float(tau), _check(H, "H", _F32),
                                 _check(route, "route", _I32, True), ws.ptr, ws.nbytes, _stream(stream))
    _raise(st, "wf_lmhead_entropy")
    return H, route


def wf_set_wait_timeout_ns(ns: int) -> None:
    lib().wf_set_wait_timeout_ns(int(ns))


def wf_probe_bounded_wait(timeout_ns: int, ws: Workspace, stream=None) -> None:
    _raise(lib().wf_probe_bounded_wait(int(timeout_ns), ws.ptr, ws.nbytes, _stream(stream)), "wf_probe_bounded_wait")


def wf_lmhead_argmax(hidden, W, ws: Workspace, ids=None, maxlogit=None, stream=None):
    P, d = hidden.shape
    V = W.shape[0]
    if ids is None:
        ids = torch.empty(P, dtype=torch.int32, device=hidden.device)
    st = lib().wf_lmhead_argmax(_check(hidden, "hidden", _BF16), _check(W, "W", _BF16), P, d, V,
                                _check(ids, "ids", _I32), _check(maxlogit, "maxlogit", _F32, True), ws.ptr, ws.nbytes,
                                _stream(stream))
    _raise(st, "wf_lmhead_argmax")
    return ids


def wf_lmhead_argmax_noalloc(hidden, W, ids=None, maxlogit=None, stream=None):
    """The LM-head argmax without a workspace (scratch in a fixed array inside the
    library), for callers that cannot allocate device memory.  Calls on one device
    share that array: do not let them overlap on the GPU."""
    P, d = hidden.shape
    V = W.shape[0]
    if ids is None:
        ids = torch.empty(P, dtype=torch.int32, device=hidden.device)
    st = lib().wf_lmhead_argmax_noalloc(_check(hidden, "hidden", _BF16), _check(W, "W", _BF16), P, d, V,
                                        _check(ids, "ids", _I32), _check(maxlogit, "maxlogit", _F32, True),
                                        _stream(stream))
    _raise(st, "wf_lmhead_argmax_noalloc")
    return ids


def wf_noalloc_read_device_error(clear: bool = True, stream=None):
    """(code, info) left on the device by the last wf_lmhead_argmax_noalloc call."""
    code, info = _i32(0), _i32(0)
    _raise(lib().wf_noalloc_read_device_error(ctypes.byref(code), ctypes.byref(info), int(clear), _stream(stream)),
           "wf_noalloc_read_device_error")
    return code.value, info.value


def wf_build_tree(tid, lp, N: int, ws: Workspace, parent=None, token=None, score=None, depth=None, stream=None):
    """EAGLE-3 draft tree from per-step, per-slot top-k children -> (parent, token, score, depth) [B, N].
    Outputs not given are allocated."""
    B, D, k, _ = tid.shape
    dev = tid.device
    parent = torch.empty((B, N), dtype=torch.int32, device=dev) if parent is None else parent
    token = torch.empty((B, N), dtype=torch.int32, device=dev) if token is None else token
    score = torch.empty((B, N), dtype=torch.float32, device=dev) if score is None else score
    depth = torch.empty((B, N), dtype=torch.int32, device=dev) if depth is None else depth
    for name, t_, dt in (("parent", parent, _I32), ("token", token, _I32), ("score", score, _F32),
                         ("depth", depth, _I32)):
        if t_.numel() < B * N:
            raise ValueError(f"{name}: needs {B * N} elements")
        _check(t_, name, dt)
    st = lib().wf_build_tree(_check(tid, "tid", _I32), _check(lp, "lp", _F32), B, D, k, N, parent.data_ptr(),
                             token.data_ptr(), score.data_ptr(), depth.data_ptr(), ws.ptr, ws.nbytes, _stream(stream))
    _raise(st, "wf_build_tree")
    return parent, token, score, depth


def wf_accepted_rows(n_accept, path, pos_off, hidden=None, acc_rows=None, acc_off=None, hidden_out=None,
                     stream=None):
    """Kept rows of each sequence (root + accepted path), their packed offsets and,
    if ``hidden`` is given, the packed hidden states of those rows.  Outputs not
    given are allocated; a ``hidden_out`` not given is sized by a host read of
    n_accept (pass one with room for B * (path stride + 1) rows to stay on the
    stream, e.g. inside a CUDA graph)."""
    B, ps = path.shape
    dev = n_accept.device
    acc_rows = torch.empty((B, ps + 1), dtype=torch.int32, device=dev) if acc_rows is None else acc_rows
    acc_off = torch.empty(B + 1, dtype=torch.int32, device=dev) if acc_off is None else acc_off
    if acc_rows.numel() < B * (ps + 1) or acc_off.numel() < B + 1:
        raise ValueError("acc_rows needs B * (path stride + 1) elements and acc_off B + 1")
    out = hidden_out
    d = 0
    if hidden is not None:
        d = hidden.shape[1]
        if out is not None and (out.dim() != 2 or out.shape[1] != d or out.shape[0] < B * (ps + 1)):
            raise ValueError("hidden_out needs room for B * (path stride + 1) rows of d columns")
        if out is None:
            total = int(n_accept.clamp(min=-1).add(1).sum().item())   # host read of the packed size
            out = torch.empty((max(total, 1), d), dtype=hidden.dtype, device=dev)
    st = lib().wf_accepted_rows(_check(n_accept, "n_accept", _I32), _check(path, "path", _I32), ps,
                                _check(pos_off, "pos_off", _I32), B, _check(acc_rows, "acc_rows", _I32),
                                _check(acc_off, "acc_off", _I32), _check(hidden, "hidden", _BF16, True), d,
                                _check(out, "hidden_out", _BF16, True), _stream(stream))
    _raise(st, "wf_accepted_rows")
    return acc_rows, acc_off, out


def _verify_outputs(B, path_stride, device, n_accept, bonus, last_pos, path):
    mk = lambda: torch.empty(B, dtype=torch.int32, device=device)  # noqa: E731
    n_accept = mk() if n_accept is None else n_accept
    bonus = mk() if bonus is None else bonus
    last_pos = mk() if last_pos is None else last_pos
    if path is None and path_stride > 0:
        path = torch.empty((B, path_stride), dtype=torch.int32, device=device)
    return n_accept, bonus, last_pos, path


def wf_verify_chain(g, draft, pos_off, node_off, ws: Workspace, path_stride: int = 0, n_accept=None, bonus=None,
                    last_pos=None, path=None, stream=None):
    B = pos_off.numel() - 1
    n_accept, bonus, last_pos, path = _verify_outputs(B, path_stride, g.device, n_accept, bonus, last_pos, path)
    st = lib().wf_verify_chain(_check(g, "g", _I32), _check(draft, "draft", _I32), _check(pos_off, "pos_off", _I32),
                               _check(node_off, "node_off", _I32), B, path_stride, _check(n_accept, "n_accept", _I32),
                               _check(bonus, "bonus", _I32), _check(last_pos, "last_pos", _I32),
                               _check(path, "path", _I32, True), ws.ptr, ws.nbytes, _stream(stream))
    _raise(st, "wf_verify_chain")
    return n_accept, bonus, last_pos, path


def wf_verify_tree(g, tok, parent, node_off, pos_off, ws: Workspace, path_stride: int = 0, n_accept=None,
                   bonus=None, last_pos=None, path=None, stream=None):
    B = pos_off.numel() - 1
    n_accept, bonus, last_pos, path = _verify_outputs(B, path_stride, g.device, n_accept, bonus, last_pos, path)
    st = lib().wf_verify_tree(_check(g, "g", _I32), _check(tok, "tok", _I32), _check(parent, "parent", _I32),
                              _check(node_off, "node_off", _I32), _check(pos_off, "pos_off", _I32), B, path_stride,
                              _check(n_accept, "n_accept", _I32), _check(bonus, "bonus", _I32),
                              _check(last_pos, "last_pos", _I32), _check(path, "path", _I32, True), ws.ptr,
                              ws.nbytes, _stream(stream))
    _raise(st, "wf_verify_tree")
    return n_accept, bonus, last_pos, path


def wf_router_mlp(hidden, rows, W1, b1, w2, b2: float, tau: float, ws: Workspace, delta_al=None, route=None,
                  stream=None):
    B = rows.numel()
    m, d = W1.shape
    if delta_al is None:
        delta_al = torch.empty(B, dtype=torch.float32, device=hidden.device)
    if route is None:
        route = torch.empty(B, dtype=torch.int32, device=hidden.device)
    st = lib().wf_router_mlp(_check(hidden, "hidden", _BF16), _check(rows, "rows", _I32), B, d, m,
                             _check(W1, "W1", _F32), _check(b1, "b1", _F32), _check(w2, "w2", _F32), float(b2),
                             float(tau), _check(delta_al, "delta_al", _F32), _check(route, "route", _I32), ws.ptr,
                             ws.nbytes, _stream(stream))
    _raise(st, "wf_router_mlp")
    return delta_al, route


def wf_draft_topk(x, Wd, d2t, k: int, ws: Workspace, draft_ids=None, tids=None, vals=None, lse=None,
                  stream=None):
    """-> (draft_ids, tids, vals); pass ``lse`` (a [B] fp32 tensor) to also receive
    each row's log-sum-exp over the draft vocabulary."""
    B, d = x.shape
    Vd = Wd.shape[0]
    dev = x.device
    draft_ids = torch.empty((B, k), dtype=torch.int32, device=dev) if draft_ids is None else draft_ids
    tids = torch.empty((B, k), dtype=torch.int32, device=dev) if tids is None else tids
    vals = torch.empty((B, k), dtype=torch.float32, device=dev) if vals is None else vals
    st = lib().wf_draft_topk(_check(x, "x", _BF16), _check(Wd, "Wd", _BF16), _check(d2t, "d2t", _I32), B, d, Vd, k,
                             _check(draft_ids, "draft_ids", _I32), _check(tids, "tids", _I32),
                             _check(vals, "vals", _F32), _check(lse, "lse", _F32, True), ws.ptr, ws.nbytes,
                             _stream(stream))
    _raise(st, "wf_draft_topk")
    return draft_ids, tids, vals


def wf_lmhead_draft_topk(hidden, W, x, Wd, d2t, k: int, ws: Workspace, ids=None, maxlogit=None, draft_ids=None,
                         tids=None, vals=None, lse=None, stream=None):
    """Target argmax over the rows of hidden and draft top-k over the rows of x
    in one weight sweep (P, B <= 128, or P > 128 and B <= 256)."""
    P, d = hidden.shape
    V = W.shape[0]
    B = x.shape[0]
    Vd = Wd.shape[0]
    if x.shape[1] != d or W.shape[1] != d or Wd.shape[1] != d:
        raise ValueError("hidden, W, x and Wd must share the hidden size d")
    dev = hidden.device
    ids = torch.empty(P, dtype=torch.int32, device=dev) if ids is None else ids
    draft_ids = torch.empty((B, k), dtype=torch.int32, device=dev) if draft_ids is None else draft_ids
    tids = torch.empty((B, k), dtype=torch.int32, device=dev) if tids is None else tids
    vals = torch.empty((B, k), dtype=torch.float32, device=dev) if vals is None else vals
    st = lib().wf_lmhead_draft_topk(_check(hidden, "hidden", _BF16), _check(W, "W", _BF16), P, d, V,
                                    _check(ids, "ids", _I32), _check(maxlogit, "maxlogit", _F32, True),
                                    _check(x, "x", _BF16), _check(Wd, "Wd", _BF16), _check(d2t, "d2t", _I32), B, Vd,
                                    k, _check(draft_ids, "draft_ids", _I32), _check(tids, "tids", _I32),
                                    _check(vals, "vals", _F32), _check(lse, "lse", _F32, True), ws.ptr, ws.nbytes,
                                    _stream(stream))
    _raise(st, "wf_lmhead_draft_topk")
    return ids, draft_ids, tids, vals


class LogprobsWorkspace(Workspace):
    """Workspace of wf_lmhead_logprobs for P rows of d, V ids, lists of S given tokens and k alternatives.  Those
    calls take no other workspace, and other calls not this one."""

    def __init__(self, P: int, d: int, V: int, S: int = 0, k: int = 0, device=None, stream=None):
        self.nbytes = int(lib().wf_logprobs_workspace_bytes(P, d, V, S, k))
        if self.nbytes == 0:
            raise ValueError("log-probability shapes outside the library's range")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        # only its control block has to be zero
        _raise(lib().wf_workspace_init(self.buf.data_ptr(), 256, _stream(stream)), "wf_workspace_init")


class Logprobs(NamedTuple):
    """What wf_lmhead_logprobs returns; None where it was not asked for."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    H: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


def _own_ws(ws, kind, dev):
    if type(ws) is not kind:
        raise ValueError(f"ws must be a {kind.__name__}")
    if ws.buf.get_device() != dev:
        raise ValueError(f"ws must be on cuda:{dev}")
    return ws.buf.data_ptr(), ws.nbytes


def _shaped(t, name, shape, dtypes, dev):
    """Address of a dense tensor of this shape on CUDA device number dev."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if t.dtype not in dtypes or not t.is_contiguous():
        return _check(t, name, dtypes)
    return t.data_ptr() or _check(t, name, dtypes)


def _head(x, W, names):
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"{names[0]} must be [rows, d] and {names[1]} [ids, d]")
    xp, dev = _check(x, names[0], _BF16), x.get_device()
    return xp, _shaped(W, names[1], W.shape, _BF16, dev), dev


def wf_lmhead_logprobs(hidden, W, ws: LogprobsWorkspace, tok=None, k: int = 0, temperature: float = 1.0,
                       with_entropy: bool = False, logp=None, lse=None, H=None, top_ids=None, top_logp=None,
                       stream=None) -> Logprobs:
    """Log-probabilities of given tokens tok [P] or [P, S] (-1: none) under softmax(hidden W^T / temperature), the
    log-sum-exp, the entropy (with_entropy, or H given) and the k best alternatives of each row.  Outputs not given
    are allocated."""
    hp, Wp, dev = _head(hidden, W, ("hidden", "W"))
    (P, d), V = hidden.shape, W.shape[0]
    S = tp = 0
    if tok is not None:
        shape = tok.shape
        S = 1 if len(shape) == 1 else shape[1] if len(shape) == 2 else 0
        if not 1 <= S <= WF_MAX_LISTED or shape[0] != P:
            raise ValueError(f"tok must be [P] or [P, S], S up to {WF_MAX_LISTED}")
        tp = _shaped(tok, "tok", shape, _I32, dev)
    # (pieces of one allocation would take longer: a view costs most of what an allocation does, and one of a given
    # shape twice what one like another tensor does)
    new, like, fp32, on = torch.empty, torch.empty_like, torch.float32, hidden.device
    lp = Hp = idp = tlp = 0
    if tok is None:
        logp = None
    elif logp is None:
        logp = like(tok, dtype=fp32)
        lp = logp.data_ptr()
    else:
        lp = _shaped(logp, "logp", shape, _F32, dev)
    if lse is None:
        lse = new(P, dtype=fp32, device=on)
        lsep = lse.data_ptr()
    else:
        lsep = _shaped(lse, "lse", (P,), _F32, dev)
    if H is not None:
        Hp = _shaped(H, "H", (P,), _F32, dev)
    elif with_entropy:
        H = like(lse)
        Hp = H.data_ptr()
    if k <= 0:
        top_ids = top_logp = None
    else:
        if top_ids is None:
            top_ids = new(P, k, dtype=torch.int32, device=on)
            idp = top_ids.data_ptr()
        else:
            idp = _shaped(top_ids, "top_ids", (P, k), _I32, dev)
        if top_logp is None:
            top_logp = like(top_ids, dtype=fp32)
            tlp = top_logp.data_ptr()
        else:
            tlp = _shaped(top_logp, "top_logp", (P, k), _F32, dev)
    args = _LOGPROBS.pack(hp, Wp, P, d, V, temperature, tp, S, k, lp, lsep, Hp, idp, tlp)
    st = (_lib or lib()).wf_lmhead_logprobs(args, *_own_ws(ws, LogprobsWorkspace, dev), _stream(stream))
    if st:
        _raise(st, "wf_lmhead_logprobs")
    return Logprobs(logp, lse, H, top_ids, top_logp)


class DistillWorkspace(Workspace):
    """Workspace of wf_draft_distill and wf_draft_distill_grad for N rows of d, Vd draft ids and k alternatives of the
    teacher.  Those calls take no other workspace, and other calls not this one."""

    def __init__(self, N: int, d: int, Vd: int, k: int, device=None, stream=None):
        self.nbytes = int(lib().wf_distill_workspace_bytes(N, d, Vd, k))
        if self.nbytes == 0:
            raise ValueError("distillation shapes outside the library's range")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        # only its control block has to be zero
        _raise(lib().wf_workspace_init(self.buf.data_ptr(), 256, _stream(stream)), "wf_workspace_init")


def distill_logits(N: int, Vd: int, device=None):
    """A buffer for the logits that wf_draft_distill keeps for the gradients: [N, Vd rounded up to 4] fp32."""
    return torch.empty((N, (Vd + 3) // 4 * 4), dtype=torch.float32, device=device or "cuda")


def _distill(fn, x, Wd, tid, tlogit, t2d, temperature, z, lse, loss, gloss, dx, dWd, ws, stream):
    xp, wp, dev = _head(x, Wd, ("x", "Wd"))
    (N, d), Vd = x.shape, Wd.shape[0]
    shape, V, ldz = tid.shape, 0, 0
    if len(shape) != 2 or shape[0] != N or not 1 <= shape[1] <= WF_MAX_LISTED:
        raise ValueError(f"tid must be [N, k], k up to {WF_MAX_LISTED}")
    if z is not None:
        if z.dim() != 2 or z.shape[0] != N or z.shape[1] < Vd or z.shape[1] % 4:
            raise ValueError("z must be [N, ldz], ldz a multiple of 4 from Vd on")
        ldz = z.shape[1]
    if t2d is not None:
        V = t2d.numel()
        if t2d.dim() != 1 or V == 0:
            raise ValueError("t2d must be [V]")
    args = _DISTILL.pack(xp, wp, N, d, Vd, _shaped(tid, "tid", shape, _I32, dev),
                         _shaped(tlogit, "tlogit", shape, _F32, dev), shape[1],
                         _shaped(t2d, "t2d", t2d.shape, _I32, dev) if V else 0, V, temperature,
                         _shaped(z, "z", z.shape, _F32, dev) if ldz else 0, ldz, _shaped(lse, "lse", (N,), _F32, dev),
                         _shaped(loss, "loss", (N,), _F32, dev) if loss is not None else 0,
                         _shaped(gloss, "gloss", (N,), _F32, dev) if gloss is not None else 0,
                         _shaped(dx, "dx", x.shape, _BF16, dev) if dx is not None else 0,
                         _shaped(dWd, "dWd", Wd.shape, _BF16, dev) if dWd is not None else 0)
    st = getattr(_lib or lib(), fn)(args, *_own_ws(ws, DistillWorkspace, dev), _stream(stream))
    if st:
        _raise(st, fn)


def wf_draft_distill(x, Wd, tid, tlogit, ws: DistillWorkspace, t2d=None, temperature: float = 1.0, z=None, loss=None,
                     lse=None, stream=None):
    """Distillation loss of the draft head against a teacher's top logits -> (loss [N], lse [N]).

    x [N, d], Wd [Vd, d] bf16; tid, tlogit [N, k]: the teacher's alternatives (-1: none), target ids if t2d [V] is
    given.  z (distill_logits) keeps the logits for wf_draft_distill_grad."""
    if loss is None:
        loss = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    if lse is None:
        lse = torch.empty_like(loss)
    _distill("wf_draft_distill", x, Wd, tid, tlogit, t2d, temperature, z, lse, loss, None, None, None, ws, stream)
    return loss, lse


def wf_draft_distill_grad(x, Wd, tid, tlogit, z, lse, ws: DistillWorkspace, gloss=None, t2d=None,
                          temperature: float = 1.0, dx=None, dWd=None, need_dx: bool = True, need_dWd: bool = True,
                          stream=None):
    """Gradients of the distillation loss -> (dx [N, d] or None, dWd [Vd, d] or None), bf16.

    z and lse as wf_draft_distill left them; gloss [N]: the derivative of what is minimised by each row's loss (None:
    1).  The other arguments as they were there."""
    if z is None:
        raise ValueError("z is required")
    if not (need_dx or need_dWd):
        raise ValueError("neither dx nor dWd is asked for")
    if not need_dx:
        dx = None
    elif dx is None:
        dx = torch.empty_like(x)
    if not need_dWd:
        dWd = None
    elif dWd is None:
        dWd = torch.empty_like(Wd)
    _distill("wf_draft_distill_grad", x, Wd, tid, tlogit, t2d, temperature, z, lse, None, gloss, dx, dWd, ws, stream)
    return dx, dWd


class CatchupWorkspace(Workspace):
    """Workspace of wf_catchup / wf_catchup_kv for B sequences, N backlog rows and the drafter's shapes."""

    def __init__(self, B: int, N: int, din: int, H: int, G: int, D: int, device=None, stream=None):
        self.nbytes = int(lib().wf_catchup_workspace_bytes(B, N, din, H, G, D))
        if self.nbytes == 0:
            raise ValueError("catch-up shapes outside the library's range")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        _raise(lib().wf_workspace_init(self.buf.data_ptr(), self.nbytes, _stream(stream)), "wf_workspace_init")


class Catchup:
    """One KV-only catch-up call (wf_catchup, or wf_catchup_kv with kv_only) over
    device tensors, repeatable and capturable in a CUDA graph.  u [N, din],
    bl_off [B+1], cache_len [B] int32; gamma [din], Wq [H*D, din], Wk / Wv
    [G*D, din], Wo [din, H*D] bf16; caches Kc / Vc [B, cap, G*D] bf16 (updated
    in place); outputs out [B, din] and attn [B, H*D] fp32."""

    def __init__(self, u, bl_off, cache_len, gamma, Wk, Wv, Kc, Vc, G: int, Wq=None, Wo=None, eps: float = 1e-6,
                 theta: float = 1e4, kv_only: bool = False, with_attn: bool = True):
        N, din = u.shape
        B = bl_off.numel() - 1
        D = Wk.shape[0] // G
        H = Wq.shape[0] // D if Wq is not None else G
        if Kc.shape != Vc.shape or Kc.dim() != 3 or Kc.shape[0] != B or Kc.shape[2] != G * D:
            raise ValueError("caches must be [B, cap, G*D]")
        if Wk.shape != (G * D, din) or Wv.shape != Wk.shape or gamma.numel() != din:
            raise ValueError("Wk / Wv must be [G*D, din] and gamma [din]")
        if not kv_only and (Wq is None or Wo is None or Wq.shape != (H * D, din) or Wo.shape != (din, H * D)):
            raise ValueError("wf_catchup needs Wq [H*D, din] and Wo [din, H*D]")
        dev = u.device
        self.kv_only = kv_only
        self.out = None if kv_only else torch.empty((B, din), dtype=torch.float32, device=dev)
        self.attn = None if kv_only or not with_attn else torch.empty((B, H * D), dtype=torch.float32, device=dev)
        self.ws = CatchupWorkspace(B, N, din, H, G, D, device=dev)
        self.tensors = (u, bl_off, cache_len, gamma, Wq, Wk, Wv, Wo, Kc, Vc)   # kept alive
        a = CatchupArgs()
        a.u = _check(u, "u", _BF16)
        a.bl_off = _check(bl_off, "bl_off", _I32)
        a.cache_len = _check(cache_len, "cache_len", _I32)
        a.B, a.N, a.din, a.H, a.G, a.D = B, N, din, H, G, D
        a.gamma = _check(gamma, "gamma", _BF16)
        a.eps, a.theta = float(eps), float(theta)
        a.Wq = _check(Wq, "Wq", _BF16, True)
        a.Wk = _check(Wk, "Wk", _BF16)
        a.Wv = _check(Wv, "Wv", _BF16)
        a.Wo = _check(Wo, "Wo", _BF16, True)
        a.Kc = _check(Kc, "Kc", _BF16)
        a.Vc = _check(Vc, "Vc", _BF16)
        a.cap = Kc.shape[1]
        a.out = _check(self.out, "out", _F32, True)
        a.attn = _check(self.attn, "attn", _F32, True)
        self.args = a

    def __call__(self, stream=None):
        fn = lib().wf_catchup_kv if self.kv_only else lib().wf_catchup
        st = fn(ctypes.byref(self.args), self.ws.ptr, self.ws.nbytes, _stream(stream))
        _raise(st, "wf_catchup_kv" if self.kv_only else "wf_catchup")
        return self.out, self.attn


class PagedCache:
    """A paged key-value cache over caller-owned device tensors (``wf_paged_cache``).

    K, V [layers, num_pages, page_size, G, D] (or without the layers: one layer),
    bf16 or float8_e4m3fn; table [B, max_pages] int32 (-1 = no page); ref
    [num_pages] int32 reference counts (wf_pages_*); k_scale / v_scale [layers, G]
    fp32 scales of an e4m3 cache.  The object keeps the tensors alive; the calls
    read and write them in place."""

    def __init__(self, K, V, table, ref=None, k_scale=None, v_scale=None):
        if K.dim() == 4 and V.dim() == 4:
            K, V = K[None], V[None]
        if K.dim() != 5 or K.shape != V.shape or K.dtype != V.dtype:
            raise ValueError("K and V must be [layers, num_pages, page_size, G, D] of one type")
        if table.dim() != 2:
            raise ValueError("table must be [B, max_pages]")
        e4m3 = K.dtype == torch.float8_e4m3fn
        types = (torch.float8_e4m3fn,) if e4m3 else _BF16
        layers, num_pages, page_size, G, D = K.shape
        for name, t_ in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t_ is not None and (not e4m3 or t_.numel() != layers * G):
                raise ValueError(f"{name}: [layers, G] fp32, of an e4m3 cache only")
        if ref is not None and ref.numel() != num_pages:
            raise ValueError("ref must be [num_pages]")
        self.K, self.V, self.table, self.ref, self.k_scale, self.v_scale = K, V, table, ref, k_scale, v_scale
        a = PagedCacheArgs()
        a.K, a.V = _check(K, "K", types), _check(V, "V", types)
        a.k_scale = _check(k_scale, "k_scale", _F32, True)
        a.v_scale = _check(v_scale, "v_scale", _F32, True)
        a.table = _check(table, "table", _I32)
        a.ref = _check(ref, "ref", _I32, True)
        a.kv_type = WF_KV_E4M3 if e4m3 else WF_KV_BF16
        a.layers, a.num_pages, a.page_size, a.G, a.D = layers, num_pages, page_size, G, D
        a.B, a.max_pages = table.shape
        self.B, self.G, self.D = a.B, a.G, a.D
        self.args = a
        self._ref = ctypes.byref(a)


class PagedWorkspace(Workspace):
    """Workspace of the wf_paged_* / wf_pages_* calls on a cache of B sequences; H query heads and max_rows rows
    a sequence as for wf_paged_attention (the other calls take any workspace of their G and D).  Those calls take no
    other workspace: elsewhere scratch may lie where they keep counters."""

    def __init__(self, B: int, H: int, G: int, D: int, max_rows: int = 1, device=None, stream=None):
        self.nbytes = int(lib().wf_paged_workspace_bytes(B, H, G, D, max_rows))
        if self.nbytes == 0:
            raise ValueError("paged cache shapes outside the library's range")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        _raise(lib().wf_workspace_init(self.buf.data_ptr(), self.nbytes, _stream(stream)), "wf_workspace_init")


def _paged(ws):
    if not isinstance(ws, PagedWorkspace):
        raise ValueError("ws must be a PagedWorkspace")
    return ws.buf.data_ptr(), ws.nbytes


def _rows(t, name, heads, D):
    """Address and row stride of [P, heads, D] bf16 rows; the rows may lie apart (a slice of a wider projection)."""
    shape, strides = t.shape, t.stride()
    if not t.is_cuda or t.dtype not in _BF16:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    if len(shape) != 3 or shape[2] != D or (heads and shape[1] != heads):
        raise ValueError(f"{name} must be [P, {heads or 'H'}, {D}]")
    if shape[0] * shape[1] == 0:
        return _placeholder(t.device), shape[1] * D
    if strides[2] != 1 or (strides[1] != D and shape[1] > 1):
        raise ValueError(f"{name}: each row's heads must lie densely")
    return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1] * D


def _lens(t, name, n, optional=False):
    """Address of n int32 numbers (None if optional and not given)."""
    if t is None and optional:
        return None
    if t is None or not t.is_cuda or t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} int32 numbers")
    return t.data_ptr() if n else _placeholder(t.device)


def wf_paged_append(cache: PagedCache, k, v, pos_off, cache_len, ws: PagedWorkspace, layer: int = 0, stream=None):
    """Store the round's keys and values (rows pos_off[b] + i of k, v [P, G, D] bf16, strided rows allowed) at
    positions cache_len[b] + i of each sequence."""
    B, G, D = cache.B, cache.G, cache.D
    kp, ks = _rows(k, "k", G, D)
    vp, vs = _rows(v, "v", G, D)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    _raise((_lib or lib()).wf_paged_append(cache._ref, layer, kp, ks, vp, vs, k.shape[0], _lens(pos_off, "pos_off", B + 1),
                                 _lens(cache_len, "cache_len", B), *_paged(ws), _stream(stream)),
           "wf_paged_append")


def wf_paged_attention(cache: PagedCache, q, pos_off, cache_len, ws: PagedWorkspace, node_off=None, kind=None,
                       parent=None, max_rows: int = 1, layer: int = 0, scale=None, out=None, lse=None,
                       with_lse: bool = False, stream=None):
    """Attention of the round's rows over the paged cache -> (out [P, H, D] bf16, lse [P, H] fp32 or None).

    q [P, H, D] bf16 (strided rows allowed), rows pos_off[b] .. pos_off[b+1]-1 of sequence b at positions
    cache_len[b] ..; single new tokens: one row each.  Chains unless parent (with node_off, and kind to mix) gives
    trees.  max_rows: most rows of a sequence.  scale: 1 / sqrt(D) if None."""
    B, D = cache.B, cache.D
    P, H = q.shape[0], q.shape[1]
    qp, stride = _rows(q, "q", 0, D)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr() if P else _placeholder(q.device)
    elif out.numel() != P * H * D:
        raise ValueError("out must be [P, H, D]")
    else:
        op = _check(out, "out", _BF16)
    if lse is not None:
        if lse.numel() != P * H:
            raise ValueError("lse must be [P, H]")
    elif with_lse:
        lse = torch.empty((P, H), dtype=torch.float32, device=q.device)
    # packed at once: setting a structure's fields one by one takes four times as long
    args = _PAGED_ATTN.pack(qp, stride, P, H, _lens(pos_off, "pos_off", B + 1), _lens(cache_len, "cache_len", B),
                            _lens(node_off, "node_off", B + 1, True) or 0, _lens(kind, "kind", B, True) or 0,
                            _check(parent, "parent", _I32, True) or 0, max_rows, layer,
                            D ** -0.5 if scale is None else scale, op,
                            0 if lse is None else _check(lse, "lse", _F32))
    st = (_lib or lib()).wf_paged_attention(cache._ref, args, *_paged(ws), _stream(stream))
    if st:
        _raise(st, "wf_paged_attention")
    return out, lse


def wf_paged_compact(cache: PagedCache, n_accept, path, cache_len, ws: PagedWorkspace, new_len=None, stream=None):
    """Move the accepted path's keys and values up behind the round's first row, in every layer -> new_len [B]
    (pass cache_len as new_len to update it in place)."""
    B = cache.B
    if path is not None and (path.dim() != 2 or path.shape[0] != B):
        raise ValueError("path must be [B, path_stride]")
    if new_len is None:
        new_len = torch.empty_like(cache_len)
    ps = path.shape[1] if path is not None else 0
    _raise((_lib or lib()).wf_paged_compact(cache._ref, _lens(n_accept, "n_accept", B), _check(path, "path", _I32, True), ps,
                                  _lens(cache_len, "cache_len", B), _lens(new_len, "new_len", B), *_paged(ws),
                                  _stream(stream)), "wf_paged_compact")
    return new_len


def wf_pages_reserve(cache: PagedCache, pos_off, cache_len, ws: PagedWorkspace, added=None, stream=None):
    """Pages for the round's rows, shared ones replaced by copies -> added [B] (pages taken, -1 = did not fit)."""
    B = cache.B
    if added is None:
        added = torch.empty_like(cache_len)
    _raise((_lib or lib()).wf_pages_reserve(cache._ref, _lens(pos_off, "pos_off", B + 1), _lens(cache_len, "cache_len", B),
                                  _lens(added, "added", B), *_paged(ws), _stream(stream)), "wf_pages_reserve")
    return added


def wf_pages_fork(cache: PagedCache, src, dst, cache_len, ws: PagedWorkspace, stream=None):
    """Sequences dst become copies of sequences src that share their pages; cache_len[dst] follows, in place."""
    n = src.numel()
    _raise((_lib or lib()).wf_pages_fork(cache._ref, _check(src, "src", _I32), _lens(dst, "dst", n), n,
                               _lens(cache_len, "cache_len", cache.B), *_paged(ws), _stream(stream)),
           "wf_pages_fork")


def wf_pages_trim(cache: PagedCache, cache_len, ws: PagedWorkspace, stream=None):
    """Give back the pages past each sequence's length (0 frees the sequence)."""
    _raise((_lib or lib()).wf_pages_trim(cache._ref, _lens(cache_len, "cache_len", cache.B), *_paged(ws),
                               _stream(stream)), "wf_pages_trim")


def _packed(spec, device):
    """One uint8 device buffer holding every (name, dtype, shape) of ``spec`` at
    256-byte aligned offsets; returns (buffer, {name: typed view})."""
    offs, total = {}, 0
    for name, dt, shape in spec:
        n = 1
        for s in shape:
            n *= s
        offs[name] = total
        total += (n * torch.empty((), dtype=dt).element_size() + 255) // 256 * 256
    buf = torch.zeros(max(total, 256), dtype=torch.uint8, device=device)
    views = {}
    for name, dt, shape in spec:
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        views[name] = buf[offs[name]:offs[name] + nbytes].view(dt).view(*shape)
    return buf, views


class Round:
    """Inputs and output buffers of wf_round, held as device tensors so the
    call can be repeated (and captured in a CUDA graph) without re-marshalling.

    The per-round inputs (hidden states, drafted tokens, tree parents, offsets,
    kinds, drafter hidden states) live in one packed device buffer and all
    outputs in another, so a host program moves a round in and out with one
    copy each (pinned_inputs / upload, pinned_outputs / download).  Weights
    (W, W1, b1, w2, Wd, d2t) stay where the caller keeps them."""

    def __init__(self, hidden, W, pos_off, node_off, tok, W1, b1, w2, b2: float, tau: float, kind=None, parent=None,
                 path_stride: int = 0, x=None, Wd=None, d2t=None, k: int = 0, with_maxlogit: bool = False,
                 router_kind: int = WF_ROUTER_NEURAL):
        dev = hidden.device
        P, d = hidden.shape
        B = pos_off.numel() - 1
        m = W1.shape[0]
        N = tok.numel()
        draft = Wd is not None
        in_spec = [("hidden", hidden.dtype, (P, d)), ("tok", torch.int32, (N,)), ("pos_off", torch.int32, (B + 1,)),
                   ("node_off", torch.int32, (B + 1,))]
        if kind is not None:
            in_spec.append(("kind", torch.int32, (B,)))
        if parent is not None:
            in_spec.append(("parent", torch.int32, (N,)))
        if draft:
            in_spec.append(("x", x.dtype, (B, d)))
        self.in_buf, views = _packed(in_spec, dev)
        for name, src in (("hidden", hidden), ("tok", tok), ("pos_off", pos_off), ("node_off", node_off),
                          ("kind", kind), ("parent", parent), ("x", x)):
            if name in views:
                views[name].copy_(src.reshape(views[name].shape))
        self.inputs = dict(W=W, W1=W1, b1=b1, w2=w2, Wd=Wd, d2t=d2t, kind=None, parent=None, x=None)
        self.inputs.update(views)
        hidden, tok, pos_off, node_off = views["hidden"], views["tok"], views["pos_off"], views["node_off"]
        kind, parent, x = views.get("kind"), views.get("parent"), views.get("x")
        out_spec = [("ids", torch.int32, (P,)), ("n_accept", torch.int32, (B,)), ("bonus", torch.int32, (B,)),
                    ("last_pos", torch.int32, (B,)), ("delta_al", torch.float32, (B,)), ("route", torch.int32, (B,))]
        if path_stride:
            out_spec.append(("path", torch.int32, (B, path_stride)))
        if with_maxlogit:
            out_spec.append(("maxlogit", torch.float32, (P,)))
        if draft:
            out_spec += [("draft_ids", torch.int32, (B, k)), ("tids", torch.int32, (B, k)),
                         ("vals", torch.float32, (B, k)), ("lse", torch.float32, (B,))]
        self.out_buf, outs = _packed(out_spec, dev)
        self.out = {name: outs.get(name) for name in ("ids", "n_accept", "bonus", "last_pos", "path", "delta_al",
                                                      "route", "maxlogit", "draft_ids", "tids", "vals", "lse")}
        self._in_spec, self._out_spec = in_spec, out_spec
        a = RoundArgs()
        a.hidden = _check(hidden, "hidden", _BF16)
        a.W = _check(W, "W", _BF16)
        a.P, a.d, a.V = P, d, W.shape[0]
        a.B = B
        a.pos_off = _check(pos_off, "pos_off", _I32)
        a.node_off = _check(node_off, "node_off", _I32)
        a.kind = _check(kind, "kind", _I32, True)
        a.tok = _check(tok, "tok", _I32)
        a.parent = _check(parent, "parent", _I32, True)
        a.path_stride = path_stride
        a.m = m
        a.W1 = _check(W1, "W1", _F32)
        a.b1 = _check(b1, "b1", _F32)
        a.w2 = _check(w2, "w2", _F32)
        a.b2, a.tau = float(b2), float(tau)
        a.x = _check(x, "x", _BF16, True)
        a.Wd = _check(Wd, "Wd", _BF16, True)
        a.d2t = _check(d2t, "d2t", _I32, True)
        a.Vd = Wd.shape[0] if Wd is not None else 0
        a.k = k if Wd is not None else 0
        a.router_kind = int(router_kind)
        for name in ("ids", "maxlogit", "n_accept", "bonus", "last_pos", "path", "delta_al", "route", "draft_ids",
                     "tids", "vals", "lse"):
            t = self.out[name]
            setattr(a, name, t.data_ptr() if t is not None else None)
        self.args = a
        self.ws = Workspace(P, B, m, a.Vd, a.k, device=dev, d=d)

    def __call__(self, stream=None):
        _raise(lib().wf_round(ctypes.byref(self.args), self.ws.ptr, self.ws.nbytes, _stream(stream)), "wf_round")
        return self.out

    # ---- host staging: one pinned buffer in, one out
    def pinned_inputs(self):
        """A pinned host copy of the packed inputs (same layout as the device buffer)."""
        return self.in_buf.cpu().pin_memory()

    def pinned_outputs(self):
        return torch.empty(self.out_buf.numel(), dtype=torch.uint8).pin_memory()

    def upload(self, host_inputs, stream=None):
        with torch.cuda.stream(stream) if stream is not None else _nullctx():
            self.in_buf.copy_(host_inputs, non_blocking=True)

    def download(self, host_outputs, stream=None):
        with torch.cuda.stream(stream) if stream is not None else _nullctx():
            host_outputs.copy_(self.out_buf, non_blocking=True)

    def capture_host_step(self, host_inputs, host_outputs):
        """Capture one host-to-host step - copy the packed inputs in from pinned
        memory, run the round, copy every output back - as a CUDA graph;
        ``replay_host_step()`` then runs it with one launch.  Call once the round
        has run eagerly at least once (its kernels are configured on first use)."""
        self._host_graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self._host_graph):
            self.in_buf.copy_(host_inputs, non_blocking=True)
            self()
            host_outputs.copy_(self.out_buf, non_blocking=True)
        return self._host_graph

    def replay_host_step(self):
        self._host_graph.replay()

    def host_views(self, host_outputs):
        """Typed views of the outputs inside a downloaded pinned buffer."""
        _, views = _packed_views(host_outputs, self._out_spec)
        return views


class _nullctx:
    def __enter__(self):
        return None

    def __exit__(self, *a):
        return False


def _packed_views(buf, spec):
    off, views = 0, {}
    for name, dt, shape in spec:
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        views[name] = buf[off:off + nbytes].view(dt).view(*shape)
        off += (nbytes + 255) // 256 * 256
    return buf, views


def wf_round(hidden, W, pos_off, node_off, tok, W1, b1, w2, b2, tau, kind=None, parent=None, path_stride=0, x=None,
             Wd=None, d2t=None, k=0, stream=None):
    """One-shot round (allocates outputs and a workspace)."""
    r = Round(hidden, W, pos_off, node_off, tok, W1, b1, w2, b2, tau, kind=kind, parent=parent,
              path_stride=path_stride, x=x, Wd=Wd, d2t=d2t, k=k)
    return r(stream)
