"""Kernels that begin while the kernel before them still runs read only through
the coherent path (no GPU: the sources are looked at).

Such a kernel waits for the one before it (grid_dependency_wait) and then reads
what that one wrote.  The read-only path (ld.global.nc: __ldg, or a load that the
compiler makes one because a kernel's parameter is const and __restrict__) is
for memory that nothing writes during the kernel's whole life, of which the
part before the wait is one."""
import os
import re

import mixed_precision_dense_sm_gb300 as lib

CSRC = os.path.join(lib.HERE, "csrc")
WAIT = "grid_dependency_wait"
NC = re.compile(r"__ldg\b|ld\.global\.nc|ld\.global\.\w+\.nc|LoadReadOnly")
RESTRICT = re.compile(r"const\s+[\w:]+(?:\s*<[^>]*>)?\s*\*\s*__restrict__")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def kernels(text):
    """(signature, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.start())
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield text[m.start():start], text[start:i]


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def test_the_kernels_are_found():
    early = [k for f in sources() for k in kernels(code(f)) if WAIT in k[1]]
    names = " ".join(sig for sig, _ in early)
    for n in ("gemm_tc_kernel", "glu_skinny_kernel", "glu_back_kernel", "glu_dbias_kernel", "glu_dot_kernel",
              "pack_pair_kernel", "unpack_pair_kernel", "forward_kernel", "backward_kernel", "sum_kernel",
              "dgate_kernel", "norm_partial_kernel", "apply_kernel", "softmax_kernel"):
        assert n in names, n


def test_no_read_only_parameters():
    bad = [(f, sig) for f in sources() for sig, body in kernels(code(f))
           if WAIT in body and RESTRICT.search(sig)]
    assert not bad, bad


def test_no_read_only_loads():
    """Nor in the functions beside them; in a file with kernels of both sorts,
    in the kernels that begin early."""
    bad = []
    for f in sources():
        ks = list(kernels(code(f)))
        early = [body for _, body in ks if WAIT in body]
        if len(early) == len(ks):
            early = [code(f)]                      # (all, or a file of functions alone)
        bad += [(f, m.group(0)) for t in early for m in NC.finditer(t)]
    assert not bad, bad


def test_softmax_promises_nothing_about_its_rows():
    """Y may be X, and the kernel before it writes X: no pointer is __restrict__."""
    assert not [f for f in sources() if f.startswith("softmax") and "__restrict__" in code(f)]
