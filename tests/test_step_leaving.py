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


def test_the_walk_of_drafts_stays_until_its_cluster_has_stopped():
    """Whoever may still be sent something by others of its cluster does not leave before a barrier of all of it."""
    text = source("pa_verify.cu")
    walk = text[text.index("verify_walk(const VerifyCall a)"):text.index("verify_pack(const VerifyCall a)")]
    leader, passes = walk[walk.index("if (warp == kWarps) {"):].split("\n        return;\n    }\n", 1)
    # the leader's last statements, and the passes': the barrier, then nothing that touches another CTA
    for part in (leader, passes):
        behind = part[part.rindex("cluster_meet()"):]
        assert "order(" not in behind and "send(" not in behind and part.rindex("cluster_meet()") > part.rindex("PA_DEV_TIMEOUT")
    # an exchange that was given up is not armed for the one after the next: its own bytes may still come
    wait = leader[leader.index("auto wait = [&]"):leader.index("auto order")]
    assert wait.index("return at;") < wait.index("mbar_arrive_expect_tx(")
