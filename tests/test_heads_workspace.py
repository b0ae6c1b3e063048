"""The heads' calls take a workspace of the device that they run on, and no other memory."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_lm_gb300 import wf


@pytest.mark.parametrize("kind", [wf.LogprobsWorkspace, wf.DistillWorkspace])
def test_the_binding_refuses_another_devices_workspace(kind):
    ws = kind.__new__(kind)
    ws.buf, ws.nbytes = torch.zeros(512, dtype=torch.uint8), 512
    with pytest.raises(ValueError, match="cuda:0"):
        wf._own_ws(ws, kind, 0)
    assert wf._own_ws(ws, kind, -1) == (ws.buf.data_ptr(), 512)
    with pytest.raises(ValueError, match=kind.__name__):
        wf._own_ws(object(), kind, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["wf_lmhead_logprobs", "wf_draft_distill", "wf_draft_distill_grad"])
def test_the_library_refuses_a_host_workspace(fn):
    dev = "cuda:0"
    x, W = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev), torch.zeros((9, 64), dtype=torch.bfloat16, device=dev)
    tid, f = torch.zeros((4, 2), dtype=torch.int32, device=dev), torch.zeros((6, 4, 12), device=dev)
    if fn == "wf_lmhead_logprobs":
        a = wf.LogprobsArgs(hidden=x.data_ptr(), W=W.data_ptr(), P=4, d=64, V=9, temperature=1.0, lse=f[0].data_ptr())
    else:
        a = wf.DistillArgs(x=x.data_ptr(), Wd=W.data_ptr(), N=4, d=64, Vd=9, tid=tid.data_ptr(), tlogit=f[1].data_ptr(),
                           k=2, temperature=1.0, z=f[2].data_ptr(), ldz=12, lse=f[3].data_ptr(), loss=f[4].data_ptr(),
                           dx=f[5].data_ptr())
    host = torch.zeros(64 << 20, dtype=torch.uint8).pin_memory()
    assert getattr(wf.lib(), fn)(ctypes.byref(a), host.data_ptr(), host.numel(), None) == 1
    torch.cuda.synchronize()
    assert not bool(host.any()) and not bool(f.any())
