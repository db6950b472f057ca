"""How the kernels around the step's attention leave when a wait has run out: nobody goes while copies, products or
other CTAs' messages may still reach what it held.  Read from the sources; no GPU is needed."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_02_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


USERS = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu")) if "tmem_dealloc(" in source(os.path.basename(f)))


@pytest.mark.parametrize("name", USERS)
def test_products_end_before_their_tensor_memory_is_freed(name):
    text = source(name)
    free = text.index("tmem_dealloc(")
    commits = [m.start() for m in re.finditer(r"commit\w*\(&?(B\.)?mma_done\b", text)]
    waits = [m.start() for m in re.finditer(r"mbar_wait_ns\(&?(B\.)?mma_done, 0, kWaitNs\)", text)]
    assert commits and waits, "no product is waited for"
    assert commits[-1] < waits[-1] < free


def test_there_are_such_kernels():
    assert {"pa_key_weights_tc.cu", "pa_packed_tc.cu", "pa_prefill_tc.cu"} <= set(USERS)
