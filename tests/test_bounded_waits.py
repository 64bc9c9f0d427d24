"""Every wait inside the tensor-core kernel without a causal rule has a bound (CPU: the source).

Its warps may give up one at a time, each when its own wait runs out, so nothing in the kernel
may wait for a fixed set of them without a limit: no named hardware barrier, and barriers of
the whole CTA only at the set-up and at the end, which every warp reaches whatever happened."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_gqa_attention_row_gb300", "csrc")


def kernel():
    text = open(os.path.join(CSRC, "dense_tc.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    begin = text.index("dense_tc_kernel(")
    return text[begin:text.index("__global__", begin)]


def test_no_hardware_barrier_within_a_role():
    body = kernel()
    assert not re.findall(r"named_bar_sync|bar\.sync|barrier\.(?:sync|cta)|__nanosleep", body)
    assert body.count("__syncthreads()") == 2
    assert body.rstrip().rfind("__syncthreads()") > body.rfind("mbar_wait")


def test_waits_are_those_with_a_limit():
    waits = set(re.findall(r"(\w*wait\w*)(?:<[^>]*>)?\(", kernel()))
    assert waits <= {"warp_wait_tc", "mbar_wait", "grid_dep_wait", "tmem_ld_wait", "tmem_st_wait",
                     "bulk_wait_group_read0"}, waits  # the last three: the thread's own accesses
