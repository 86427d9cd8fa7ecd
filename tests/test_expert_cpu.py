"""The experts' row moves on the CPU: exports and refusals (no GPU).  A call whose
arguments are accepted ends at the missing device (GEMM_ERR_LAUNCH)."""
import pytest
import torch

import mixed_precision_dense_sm_gb300 as lib

F16, BF16, F32 = lib.GEMM_F16, lib.GEMM_BF16, lib.GEMM_F32
BAD = 1
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are made up")


def sort(T=4, k=2, E=8, ids=64, ld=2, by=4, pos=64, offsets=64, order=64):
    return lib.expert_sort_raw(T, k, E, ids, ld, by, pos, offsets, order)


def test_declared():
    names = lib.declared_symbols()
    for n in ("expert_sort", "expert_gather", "expert_combine", "expert_gather_backward",
              "expert_combine_backward"):
        assert n in names and hasattr(lib.lib, n)
    text = open(lib.HEADERS[-1] if "expert" in lib.HEADERS[-1] else
                next(h for h in lib.HEADERS if "expert" in h)).read()
    assert f"#define EXPERT_MAX {lib.EXPERT_MAX}\n" in text


def test_sort_arguments():
    for good in ({}, dict(by=8), dict(order=0), dict(E=1024), dict(ld=9), dict(T=0, ids=0, pos=0),
                 dict(k=0, ld=1, ids=0, pos=0), dict(T=2 ** 29)):
        assert sort(**good) != BAD, good
    for bad in (dict(T=-1), dict(k=-1), dict(E=0), dict(E=-3), dict(E=1025), dict(ld=1), dict(by=2),
                dict(by=0), dict(ids=0), dict(ids=66), dict(ids=68, by=8), dict(pos=0), dict(pos=65),
                dict(offsets=0), dict(offsets=66), dict(order=67), dict(T=2 ** 30), dict(T=2 ** 62, k=4, ld=4)):
        assert sort(**bad) == BAD, bad


CALLS = ("expert_gather", "expert_combine", "expert_gather_backward", "expert_combine_backward")


def rows(name, T=4, k=2, D=16, n=8, a=64, lda=16, b=64, ldb=16, pos=64, c=64, ldc=16, dt=BF16, w=None):
    """a: the first input, b: a backward pass's second, c: the output."""
    args = (a or None, lda) + ((b or None, ldb) if name.endswith("backward") else ()) + (pos or None, c or None, ldc, dt)
    return lib.expert_rows_raw(name, T, k, D, n, *args, weights=w)


def weights(w=64, ldw=2, wt=F32, dw=64, lddw=2, dwt=F32):
    return lib.ExpertWeights(w or None, ldw, wt, dw or None, lddw, dwt)


@pytest.mark.parametrize("name", CALLS)
def test_rows_arguments(name):
    back = name.endswith("backward")
    for good in ({}, dict(w=weights()), dict(w=weights(dw=0)), dict(w=weights(w=0)), dict(lda=17, ldc=19),
                 dict(dt=F32), dict(dt=F16), dict(a=66, c=70), dict(T=0, pos=0), dict(k=0, pos=0),
                 dict(n=0)) + ((dict(c=0, w=weights()), dict(b=0)) if back else ()):
        assert rows(name, **good) != BAD, good
    for bad in (dict(T=-1), dict(k=-1), dict(D=-1), dict(n=-1), dict(lda=15), dict(ldc=15), dict(dt=3),
                dict(dt=-1), dict(a=0), dict(a=65), dict(c=65), dict(a=66, dt=F32), dict(pos=0),
                dict(pos=66), dict(T=2 ** 30), dict(D=2 ** 31, lda=2 ** 31, ldb=2 ** 31, ldc=2 ** 31),
                dict(n=2 ** 31), dict(w=weights(w=66)), dict(w=weights(ldw=1)),
                dict(w=weights(wt=5))) + \
            ((dict(w=weights(dw=66)), dict(w=weights(lddw=1)), dict(w=weights(dwt=9)), dict(c=0),
              dict(c=0, w=weights(dw=0)), dict(b=0, w=weights()), dict(ldb=15, w=weights()),
              dict(b=65, w=weights())) if back else (dict(c=0),)):
        assert rows(name, **bad) == BAD, bad


def test_tensors_on_the_cpu_are_refused():
    x, pos = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: lib.expert_sort(pos, 4), lambda: lib.expert_gather(x, pos),
                 lambda: lib.expert_combine(x, pos), lambda: lib.expert_gather_backward(x, pos, dX=x),
                 lambda: lib.expert_combine_backward(x, pos, dYs=x)):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            call()
