"""What may start beside what, around the heads' sweeps and products, checked in the sources (no GPU needed).

A sweep or a product takes whole SMs, its CTA pairs both SMs of a pair at once.  A kernel that waits for it must not
sit on an SM that one of its pairs still needs, so neither lets its dependents start early, and only a kernel of the
same call whose blocks fit beside it in any order is followed by one that starts early."""
import os
import re

import pytest

from speculative_decoding_verify_lm_gb300 import build as B


def source(name):
    with open(os.path.join(B.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """{name: body} of a file's kernels."""
    out = {}
    for at in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
        rest = text[at.end():]
        rest = rest[rest.index("{") + 1:]
        out[at.group(1)] = rest[:rest.index("\n}")]
    return out


ALL = {**kernels(source("wf_sweep.cu")), **kernels(source("wf_heads.cu")), **kernels(source("wf_distill.cu"))}


def test_whole_sm_kernels_let_nothing_start_early():
    for name in ("sweep_kernel", "grad_products_kernel"):
        assert "pipe_begin" in ALL[name] and "pdl_trigger" not in ALL[name]
        # every warp but the copying one, which waits inside, waits before it touches what a kernel wrote
        assert "if (warp != 0) pdl_wait();" in ALL[name]
    assert "pdl_wait();" in source("wf_pipe.cuh") and "pdl_trigger" not in source("wf_pipe.cuh")


def test_only_lists_and_the_logits_gradient_are_followed_early():
    early = {n for n, body in ALL.items() if "pdl_trigger();" in body}
    assert early == {"teacher_kernel", "logit_grad_kernel"}
    programmatic = re.compile(r"\b(launch|launch_cluster)\((\w+)")
    used = [m.group(2) for f in ("wf_sweep.cu", "wf_heads.cu", "wf_distill.cu") for m in programmatic.finditer(source(f))]
    assert sorted(used) == ["grad_products_kernel", "kernel"]
    assert "c.after_lists ? launch_cluster(kernel" in source("wf_sweep.cu")
    for name in early | {"states_merge_kernel", "dx_join_kernel"}:
        assert any("launch_plain(" + name in source(f) for f in ("wf_heads.cu", "wf_distill.cu")), name


def test_weights_are_asked_for_early_behind_the_calls_own_kernel_only():
    """A sweep asks for its first weights before it waits: it may, behind the list kernel of its call, which runs only
    when everything before it (an optimiser's step on these weights) is done."""
    api = source("wf_api.cu")
    assert api.count("after_lists") == 1
    at = api.index("after_lists")
    assert "launch_teacher(" in api[api.rindex("wf_status wf_draft_distill(", 0, at):at]


@pytest.mark.parametrize("name", ["wf_sweep.cu", "wf_distill.cu"])
def test_epilogues_wait_as_whole_warps(name):
    pipe = source("wf_pipe.cuh")
    wait = pipe[pipe.index("bool pipe_acc_wait"):]
    assert "__all_sync(0xffffffffu, there)" in wait[:wait.index("\n}")]
    assert "pipe_acc_wait(g, i)" in source(name) and "mbar_wait(" not in source(name)


def test_products_in_flight_are_waited_for():
    """When a wait gives up the CTA frees its tensor memory and leaves: products still in flight are waited for whatever
    the abort flag says, and so are copies."""
    pipe = source("wf_pipe.cuh")
    assert re.search(r"mbar_wait\(drain, 0, g\.timeout_ns, nullptr\)", pipe)
    assert re.search(r"mbar_wait\(&g\.full\[j % g\.stages\], \(j / g\.stages\) & 1, g\.timeout_ns, nullptr\)", pipe)


def test_no_read_only_promises():
    for name in ("wf_sweep.cu", "wf_heads.cu", "wf_heads.cuh", "wf_pipe.cuh", "wf_distill.cu"):
        assert "__restrict__" not in source(name) and "__ldg(" not in source(name)
