"""What a kernel may read before its dependency wait, checked in the sources
(no GPU needed).

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
