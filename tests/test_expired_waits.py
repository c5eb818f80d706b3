"""A wait that runs out in an 8-bit product: read in the source, since no test may make one run out in a kernel with copies under way.

The CTA's sums are incomplete then.  Ahead of anything that takes them (the join of a cluster) or that would leave the output as it was, the CTA
looks at its abort word and puts NaN in their place; no warp with fewer registers than the epilogue's takes part.
"""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_decoding_array_gb300", "csrc", "matmul_e4m3.cu")


def test_the_sums_of_an_aborted_cta_become_nan_ahead_of_the_join():
    s = re.sub(r"//[^\n]*", "", open(SRC).read())
    body = s[s.index("matmul_e4m3_kernel(const __grid_constant__"):]
    roles_end = body.rindex("__syncthreads();")
    tail = body[roles_end:]
    look = tail.index("if (*abort_flag && warp < S::kEpiWarps)")
    join = tail.index("ld_cluster_f4")
    first_sync = tail.index("cluster_sync()")
    assert look < first_sync < join
    marked = tail[look:first_sync]
    # a cluster's share: the whole staging area; else every tile of the CTA, or its rows' bests
    assert "reinterpret_cast<float*>(ring)[e] = nan" in marked and "kMmRows * BN" in marked
    assert "pack_best(nan" in marked and "put(q.p" in marked
    assert "__syncthreads" not in tail[len("__syncthreads();"):look]  # nothing between the roles' end and the look
