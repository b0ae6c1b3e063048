"""What a kernel may read before its dependency wait and has to wait for before
it leaves, checked in the sources (no GPU needed).

Every kernel is launched while its predecessor on the stream may still be
running.  A call's own inputs (rows, offsets, lengths, tables) can be what that
predecessor writes, so the first kernel of a call reads them behind
``pdl_wait()`` only."""
import os
import re

import pytest

from speculative_decoding_verify_lm_gb300 import build as B


def source(name):
    with open(os.path.join(B.CSRC, name)) as f:
        return f.read()


def kernel(name, kernel_name):
    """(parameters, body up to the dependency wait, the whole body) of a kernel, comments taken out."""
    text = re.sub(r"//[^\n]*", "", source(name))
    at = re.search(r"__global__[^;{]*?\b%s\(" % kernel_name, text)
    assert at, kernel_name
    params, rest = text[at.end():].split("{", 1)
    body = rest[:rest.index("\n}")]
    assert "pdl_wait();" in body, kernel_name
    return params, body[:body.index("pdl_wait();")], body


def test_the_catch_up_reads_its_inputs_behind_the_wait():
    """Compaction and forking write cache_len and attention writes rows, each straight before a catch-up."""
    params, early, whole = kernel("wf_catchup.cu", "norm_kernel")
    early = re.sub(r"prefetch_l2\([^;]*;", "", early)        # into L2 only: no value is read
    for name in ("u", "bl_off", "cache_len"):
        assert re.search(r"\b%s\b" % name, whole), name
        assert not re.search(r"\b%s\b" % name, early), f"norm_kernel reads {name} before its wait"
        # nor may the compiler take it for constant while the kernel before still writes it
        assert not re.search(r"__restrict__ %s\b" % name, params), name


INPUTS = r"\b(p\.|c\.)?(q|k|v|pos_off|cache_len|table|ref|n_accept|path|node_off|kind|parent|src|dst|copies|n_copies)\b"


@pytest.mark.parametrize("name,kernel_name", [
    ("wf_paged.cu", "append_kernel"), ("wf_paged.cu", "compact_kernel"), ("wf_paged.cu", "reserve_kernel"),
    ("wf_paged.cu", "page_copy_kernel"), ("wf_paged.cu", "fork_kernel"), ("wf_paged.cu", "trim_kernel"),
    ("wf_paged_token.cu", "paged_token_kernel"), ("wf_paged_rounds.cu", "paged_rounds_kernel"),
    ("wf_paged_rounds.cu", "rounds_join_kernel"),
])
def test_paged_kernels_read_and_promise_nothing_before_the_wait(name, kernel_name):
    """Compaction in place, then trim: what one writes the next reads, and was launched meanwhile."""
    params, early, whole = kernel(name, kernel_name)
    assert not re.search(INPUTS, early), re.search(INPUTS, early)
    assert "__restrict__" not in params


@pytest.mark.parametrize("name", ["wf_paged.cu", "wf_paged_token.cu", "wf_paged_rounds.cu", "wf_paged.cuh"])
def test_paged_kernels_take_only_scales_for_constant(name):
    """Loads that assume that nobody writes meanwhile are left to the model's scales."""
    text = re.sub(r"//[^\n]*", "", source(name))
    assert "__restrict__" not in text
    for arg in re.findall(r"__ldg\(([^)]*)\)", text):
        assert re.match(r"(p\.[kv]_scale|sc) \+", arg), arg


def test_the_lanes_of_a_warp_give_up_together():
    """The copying warps exchange values between their lanes: a wait that gives up has to end for all of them or for
    none, or those that stay wait for those that left without a limit."""
    for name in ("wf_paged_rounds.cu", "wf_paged_token.cu"):
        text = re.sub(r"//[^\n]*", "", source(name))
        text = text.replace("whole_warp(", "__all_sync(0xffffffffu, ")
        for barrier in ("piece_free", "q_empty", "s_empty"):
            for wait in re.finditer(r"mbar_wait\(&%s\b" % barrier, text):
                before = text[:wait.start()]
                assert "__all_sync" in before[before.rindex("\n", 0, before.rindex("\n")):] , (name, barrier)
        calls = [m.start() for m in re.finditer(r"(?<!auto )\bplace_free\(at\)", text)]
        for at in calls:
            assert text[:at].endswith("__all_sync(0xffffffffu, "), name


@pytest.mark.parametrize("name", ["wf_gemm_select.cu", "wf_catchup.cu", "wf_paged_rounds.cu"])
def test_a_wait_that_gives_up_lets_its_products_complete(name):
    """When a wait gives up the CTA frees its tensor memory and leaves.  Products of the tensor cores still in flight
    would go on reading its shared memory: they are waited for on a barrier that they commit to, whatever the abort
    flag says."""
    text = re.sub(r"//[^\n]*", "", source(name))
    commits = set(re.findall(r"umma_commit\(&?(\w+)", text))
    drained = set(re.findall(r"mbar_wait\(&?(\w+)(?:\[\w+\])?, \w+, p\.timeout_ns, nullptr\)", text))
    assert commits & drained, (commits, drained)
