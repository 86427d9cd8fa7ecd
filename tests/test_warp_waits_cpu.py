"""Warps that wait and then act together (no GPU: the sources are looked at).

A bounded wait may end differently for two lanes of a warp, at the limit.  Where
all lanes wait, they vote before anything collective (a load from tensor memory, a
full-mask barrier): a lane that left alone would leave the others waiting."""
import os
import re

import mixed_precision_dense_sm_gb300 as lib


def body(text, head):
    """The block that follows the first `head`."""
    start = text.index("{", text.index(head))
    depth, i = 1, start + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[start:i]


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(lib.HERE, "csrc", name)).read())


def test_the_updates_epilogue_votes():
    text = body(source("ortho_kern.cuh"), "bool ortho_epilogue(")
    assert len(re.findall(r"\bortho_wait\(", text)) == 1
    assert re.search(r"if \(!__all_sync\(0xffffffffu, ortho_wait\([^;]*\)\)\) return false;", text)


def test_what_one_lane_acquired_the_warp_reads_behind_a_barrier():
    """ortho_ready acquires with one lane; a shuffle hands its answer on and orders no
    memory, __syncwarp does."""
    text = source("ortho_kern.cuh")
    calls = [m for m in re.finditer(r"if \(lane == 0\) \w+ = ortho_ready\(", text)]
    assert len(calls) == 1
    rest = text[calls[0].end():]
    between = rest[:rest.index("ortho_epilogue<")]
    assert re.search(r"__shfl_sync\(.*__syncwarp\(\);", between, flags=re.S)


def test_the_gemm_epilogue_votes():
    """Between the wait for the accumulator and the collective loads: over all epilogue
    warps where they share barriers, else over the warp."""
    text = source("gemm_tc.cuh")
    waits = [m for m in re.finditer(r"wait_or_abort\(&acc_full", text)]
    assert len(waits) == 1
    rest = text[waits[0].start():]
    assert re.search(r"ok = epilogue_all\(ok\);\s*else ok = __all_sync\(0xffffffffu, ok\);\s*if \(!ok\)",
                     rest[:rest.index("tc_fence_after_sync")])
