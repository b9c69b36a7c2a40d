"""What the cache's kernels and binding rest on, checked without a GPU."""
import os
import re

from ternary_weight_gb300 import _build


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return f.read()


def test_softmax_warps_fence_behind_every_wait_for_a_product():
    """Tensor memory that a product has read or written is touched only behind a fence after the wait for it:
    without the fence nothing orders the access. (The waits of the issuing warp stand before its own
    products, with one fence for several waits; here each has its own.)"""
    softmax = re.search(r"= softmax =.*?= expansion =", source("kv4_prompt.cu"), re.S).group(0)
    waits = re.findall(r"wait\(&(?:pv_done|s_full)\[tile\].*?;\n\s*__syncwarp\(\);\n\s*([^\n]*)", softmax)
    assert len(waits) == len(re.findall(r"wait\(&(?:pv_done|s_full)", softmax)) == 4
    assert all(w.startswith("tc_fence_after();") for w in waits), waits
