"""The experts' sort and row moves refuse outputs that share memory with inputs or each
other, and take ones that only lie between each other's rows (the predicate itself:
tests/host/overlap.cpp)."""
import pytest
import torch

import expert_ref as ex

pytestmark = pytest.mark.gpu

T, K, D = 40, 3, 64


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def problem():
    gen = torch.Generator().manual_seed(1)
    pos = ex.sort(torch.randint(0, 5, (T, K), generator=gen), 5)[0].cuda()
    x, rows, w = (torch.randn(*s, generator=gen).cuda() for s in ((T, D), (T * K, D), (T, K)))
    return pos, x, rows, w


def test_refused(lib):
    pos, x, rows, w = problem()
    ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    both = torch.zeros(T * K + 6, dtype=torch.int32, device="cuda")
    big = torch.randn(2 * T * K, D, device="cuda")
    over_w = torch.zeros(T * K * D, device="cuda")
    i32 = pos.view(torch.float32)
    refused = [
        lambda: lib.expert_sort(ids, 5, pos=ids),
        lambda: lib.expert_sort(ids, 5, order=ids.view(-1)),
        lambda: lib.expert_sort(ids, 5, offsets=ids.view(-1)[:6]),
        lambda: lib.expert_sort(ids, 5, order=both[:T * K], offsets=both[T * K - 1:T * K + 5]),
        lambda: lib.expert_gather(big[:T], pos, Xs=big[T - 1:T - 1 + T * K]),
        lambda: lib.expert_gather(big[5:5 + T], pos, Xs=big[:T * K]),
        lambda: lib.expert_combine(big[:T * K], pos, Y=big[:T]),
        lambda: lib.expert_combine(big[:T * K], pos, Y=big[T * K - 1:T * K - 1 + T]),
        lambda: lib.expert_combine(rows, pos, over_w[:T * K].view(T, K), Y=over_w[:T * D].view(T, D)),
        lambda: lib.expert_combine(rows[:, :K], pos, Y=i32),
        lambda: lib.expert_gather_backward(rows, pos, w, x, dX=x, dweight=torch.empty_like(w)),
        lambda: lib.expert_gather_backward(rows, pos, w, x, dweight=w),
        lambda: lib.expert_gather_backward(rows, pos, w, x, dX=over_w[:T * D].view(T, D), dweight=over_w[:T * K].view(T, K)),
        lambda: lib.expert_combine_backward(big[:T], pos, w, dYs=big[:T * K]),
        lambda: lib.expert_combine_backward(x, pos, w, big[:T * K], dYs=big[1:1 + T * K], dweight=torch.empty_like(w)),
        lambda: lib.expert_combine_backward(x, pos, w, rows, dweight=rows.view(-1)[:T * K].view(T, K)),
    ]
    for n, call in enumerate(refused):
        with pytest.raises(lib.GemmError) as e:
            call()
        assert e.value.status == 1, n
    # in place with another leading dimension
    wide = torch.randn(T * K, 2 * D, device="cuda")
    st = lib.expert_rows_raw("expert_combine_backward", T, K, D, T * K, x.data_ptr(), D, wide.data_ptr(), 2 * D,
                             pos.data_ptr(), wide.data_ptr(), D, lib.GEMM_F32,
                             weights=lib.ExpertWeights(w.data_ptr(), K, lib.GEMM_F32, torch.empty_like(w).data_ptr(), K,
                                                       lib.GEMM_F32))
    assert st == 1


def test_taken(lib):
    pos, x, rows, w = problem()
    # tokens and rows as columns of one buffer
    buf = torch.zeros(T * K, 2 * D, device="cuda")
    buf[:T, :D] = x
    want = lib.expert_gather(x, pos, w)
    assert torch.equal(lib.expert_gather(buf[:T, :D], pos, w, Xs=buf[:, D:]), want)
    assert torch.equal(buf[:T, :D], x)
    # results in every other row
    buf = torch.zeros(2 * T * K, D, device="cuda")
    buf[::2] = rows
    want = lib.expert_combine(rows, pos, w)
    assert torch.equal(lib.expert_combine(buf[::2], pos, w, Y=buf[1:2 * T:2]), want)
    assert torch.equal(buf[::2], rows)
    # gradients of the weights in the padding of the weights
    pair = torch.zeros(T, 2 * K, device="cuda")
    pair[:, :K] = w
    dw = torch.empty_like(w)
    lib.expert_gather_backward(rows, pos, w, x, dweight=dw)
    lib.expert_gather_backward(rows, pos, pair[:, :K], x, dweight=pair[:, K:])
    assert torch.equal(pair[:, K:], dw) and torch.equal(pair[:, :K], w)
    # in place over Ys, and one row of any leading dimension
    inplace, dys = rows.clone(), torch.zeros_like(rows)
    lib.expert_combine_backward(x, pos, w, rows, dYs=dys, dweight=dw)
    lib.expert_combine_backward(x, pos, w, inplace, dYs=inplace, dweight=torch.empty_like(dw))
    assert torch.equal(inplace, dys)
    # what lies side by side
    ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    mem = torch.zeros(2 * T * K + 6, dtype=torch.int32, device="cuda")
    got = lib.expert_sort(ids, 5, pos=mem[:T * K].view(T, K), order=mem[T * K:2 * T * K], offsets=mem[2 * T * K:])
    for a, b in zip(got, ex.sort(ids.cpu(), 5)):
        assert torch.equal(a.cpu(), b)
