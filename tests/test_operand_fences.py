"""Operands of tcgen05.mma that a kernel writes to shared memory itself (CPU, on the sources).

The tensor cores read shared memory through the async proxy.  A barrier alone does not order ordinary stores before
such reads: each writing thread needs a proxy fence first.  Without it a kernel's results are wrong only when its first
product overtakes the stores, which no run shows reliably, so the sources are looked at instead."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_kvc_gb300", "csrc")
COMMENT = re.compile(r"//[^\n]*|/\*.*?\*/", re.S)


def code(path):
    with open(path) as f:
        return COMMENT.sub("", f.read())


SOURCES = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))) if os.path.basename(p) != "kvc_tc.cuh"
           and re.search(r"\btc_mma_\w+\(", code(p)) and "sts128" in code(p)]


def test_the_kernels_are_found():
    assert {os.path.basename(p) for p in SOURCES} >= {"kvc_select_tc.cu", "kvc_prefill_tc.cuh", "kvc_decode_tc.cuh"}


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_written_operands_are_fenced(path):
    """Stores, then the writers' fence, then the CTA's barrier or the warp's announcement: in this order somewhere."""
    events = re.findall(r"sts128|fence_proxy_async_smem\(\)|__syncthreads\(\)|mbar_arrive\(", code(path))
    kinds = "".join({"sts128": "w", "fence_proxy_async_smem()": "f"}.get(e, "b") for e in events)
    assert re.search("wfb", kinds), kinds
