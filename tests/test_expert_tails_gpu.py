"""GPU parity of the experts' row moves on short rows that begin on 16 bytes and end
inside a vector: each element behind the last whole vector is moved, with few threads
per token too, and by the calls without the weights' gradient."""
import pytest
import torch

import expert_ref as ex
import ffn_ref as ref
from test_expert_gpu import IDS, cpu, pitched, problem

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=IDS.get)
@pytest.mark.parametrize("D", [1, 2, 3, 5, 6, 7, 9, 11, 13, 14, 15, 21, 22, 23, 29, 30, 31, 37, 38, 39, 45, 47, 63, 71])
@pytest.mark.parametrize("T,k", [(1, 8), (5, 3), (350, 2), (40, 9)])
def test_short_rows_with_a_tail(lib, T, k, D, dtype):
    pad = -D % (4 if dtype is F32 else 8)
    for wtype, drop in ((F32, 0.0), (None, 0.3)):
        pos, x, rows, w = problem(T, k, D, dtype, wtype, drop, pad)
        p = pos.cuda()
        for m in (x, rows):
            assert m.data_ptr() % 16 == 0 and (m.stride(0) * m.element_size()) % 16 == 0

        def into(n):
            return pitched(n, D, dtype, pad)

        def check(m, buf, r, tol, what):
            ref.check(m, r, tol, what)
            m.fill_(77.0)
            assert bool((buf == 77.0).all()), f"{what}: padding"

        want = ex.out(x.cpu(), pos, cpu(w), torch.full((T * k, D), 77.0, dtype=dtype))
        for call in (lambda m: lib.expert_gather(x, p, w, Xs=m),
                     lambda m: lib.expert_combine_backward(x, p, w, dYs=m)):
            m, buf = into(T * k)
            call(m)
            check(m, buf, *want, "rows")
        want = ex.back(rows.cpu(), pos, cpu(w), D)
        for call in (lambda m: lib.expert_combine(rows, p, w, Y=m),
                     lambda m: lib.expert_gather_backward(rows, p, w, dX=m)):
            m, buf = into(T)
            call(m)
            check(m, buf, *want, "tokens")
        # with the weights' gradient, into pitched results as well
        dw = torch.empty(T, k, device="cuda")
        dots = ex.dots(x.cpu(), rows.cpu(), pos, F32)
        m, buf = into(T)
        lib.expert_gather_backward(rows, p, w, x, dX=m, dweight=dw)
        ref.check(dw, *dots, "dweight")
        check(m, buf, *want, "dX")
        m, buf = into(T * k)
        lib.expert_combine_backward(x, p, w, rows, dYs=m, dweight=dw.zero_())
        ref.check(dw, *dots, "dweight")
        check(m, buf, *ex.out(x.cpu(), pos, cpu(w), torch.full((T * k, D), 77.0, dtype=dtype)), "dYs")
