"""Kernels that are set up while the one before them still runs may share an SM with it, and with
it the SM's tensor memory. In the sources: whoever lets the next kernel in has its tensor
memory already, so that no block waits for columns that a block waiting for it holds."""
import os
import re

import pytest

import hierarchical_sparse_attention_mean_gb300 as llsa

CSRC = os.path.join(os.path.dirname(llsa.__file__), "csrc")
CALL = re.compile(r"tmem_alloc\(smem_u32|__syncthreads\(\);|close_ahead\(\);|close_wait\(\);")


def calls(name):
    """The calls of CALL in a source, comments left out, in their order."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    return [m.group(0).split("(")[0] for m in CALL.finditer(code)]


SOURCES = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and {"tmem_alloc", "close_ahead"} <= set(calls(f))]


def test_there_are_such_kernels():
    assert {"diff_fwd_tc.cu", "diff_bwd_tc.cu", "diff_bwd_wide_tc.cu", "dense_split_tc.cu", "dense_split_wide_tc.cu"} <= set(SOURCES)


@pytest.mark.parametrize("name", SOURCES)
def test_the_next_kernel_comes_in_behind_the_allocation(name):
    got = calls(name)
    kernels = [i for i, c in enumerate(got) if c == "tmem_alloc"]
    for first, end in zip(kernels, kernels[1:] + [len(got)]):
        ahead = [i for i in range(first, end) if got[i] == "close_ahead"]
        assert len(ahead) == 1 and "close_wait" in got[first:end]
        assert "__syncthreads" in got[first:ahead[0]], "close_ahead before the block has its tensor memory"
    assert "close_ahead" not in got[:kernels[0]]
