"""Calls of the experts' sort and row moves as a program makes them: long sorts and many
tokens captured and on two streams at once, one row for several choices, no choices at
all, the weights' gradient alone."""
import pytest
import torch

import expert_ref as ex
import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def ids_of(T, k, E, seed, drop=0.2):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=gen)
    ids[torch.rand(T, k, generator=gen) < drop] = -1
    return ids


def sorted_on_cpu(ids, E):
    key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
    kept = int((key < E).sum())
    order = torch.sort(key, stable=True)[1]
    pos = torch.full_like(key, -1)
    pos[order[:kept]] = torch.arange(kept)
    return pos.view(ids.shape).int()


def test_long_sort_and_ring_captured_and_on_two_streams(lib):
    """200000 slots (three launches), 20000 tokens (the ring): a graph that replays on new
    ids beside eager calls on another stream."""
    T, k, E, D = 50000, 4, 300, 256
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(T, D, generator=gen).to(BF).cuda()
    w = torch.rand(T, k, generator=gen).cuda()
    ids = [ids_of(T, k, E, s).cuda() for s in (1, 2, 3)]
    rows = torch.zeros(T * k, D, dtype=BF, device="cuda")

    def chain(i, xs):
        pos, _, order = lib.expert_sort(i, E)
        lib.expert_gather(x, pos, Xs=xs)
        return pos, order, lib.expert_combine(xs, pos, w)

    want = [[t.clone() for t in chain(i, torch.zeros_like(rows))] for i in ids]
    for i, got in zip(ids, want):
        assert torch.equal(got[0].cpu(), sorted_on_cpu(i.cpu(), E))
    fixed = ids[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(fixed, rows)
    side = torch.cuda.Stream()
    for n in (1, 2, 0):
        fixed.copy_(ids[n])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = chain(ids[(n + 1) % 3], torch.zeros_like(rows))
        torch.cuda.synchronize()
        for a, b in zip(out, want[n]):
            assert torch.equal(a, b)
        for a, b in zip(other, want[(n + 1) % 3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,k,D,rows", [(30, 3, 40, 7), (9, 10, 77, 4), (10000, 4, 512, 100)])
def test_one_row_for_several_choices(lib, T, k, D, rows):
    """What only reads the rows takes a row more than once."""
    gen = torch.Generator().manual_seed(T)
    pos = torch.randint(-1, rows, (T, k), generator=gen, dtype=torch.int32)
    ys, x, w = (torch.randn(*s, generator=gen) for s in ((rows, D), (T, D), (T, k)))
    on = (pos >= 0).double()
    picked = ys.double()[pos.clamp(min=0).long()] * on[..., None]
    part = picked * w.double()[..., None]
    e = part.abs().sum(1) * (k * ref.U32)
    y, tol = part.sum(1), e + ref.rounding(part.sum(1).abs() + e, F32)
    ref.check(lib.expert_combine(ys.cuda(), pos.cuda(), w.cuda()), y, tol, "Y")
    dx, dw = torch.empty(T, D, device="cuda"), torch.empty(T, k, device="cuda")
    lib.expert_gather_backward(ys.cuda(), pos.cuda(), w.cuda(), x.cuda(), dX=dx, dweight=dw)
    ref.check(dx, y, tol, "dX")
    prod = x.double()[:, None] * picked
    e = prod.abs().sum(2) * ((D / 32 + 22) * ref.U32)
    ref.check(dw, prod.sum(2), e + ref.rounding(prod.sum(2).abs() + e, F32), "dweight")


@pytest.mark.parametrize("T,D", [(5, 40), (20000, 1024)])
def test_no_choices(lib, T, D):
    pos = torch.empty(T, 0, dtype=torch.int32, device="cuda")
    rows = torch.full((4, D), float("nan"), dtype=BF, device="cuda")
    assert not lib.expert_combine(rows, pos).any()
    dx = torch.ones(T, D, dtype=BF, device="cuda")
    lib.expert_gather_backward(rows, pos, dX=dx)
    assert not dx.any()
    before = rows.clone()
    lib.expert_gather(dx, pos, Xs=rows)
    lib.expert_combine_backward(dx, pos, dYs=rows)
    assert bool(rows.isnan().all()) and torch.equal(before.isnan(), rows.isnan())


def test_weights_gradient_alone_of_many_tokens(lib):
    T, k, D = 12000, 5, 512
    pos = ex.sort(ids_of(T, k, 6, 4), 6)[0]
    gen = torch.Generator().manual_seed(5)
    x, rows = (torch.randn(n, D, generator=gen).to(BF).cuda() for n in (T, T * k))
    w = torch.rand(T, k, generator=gen).cuda()
    both, alone, dx = torch.empty_like(w), torch.empty_like(w), torch.empty_like(x)
    lib.expert_gather_backward(rows, pos.cuda(), w, x, dX=dx, dweight=both)
    lib.expert_gather_backward(rows, pos.cuda(), w, x, dweight=alone)
    assert torch.equal(both, alone)
    picked = rows.double()[pos.cuda().clamp(min=0).long()] * (pos.cuda() >= 0)[..., None]
    prod = x.double()[:, None] * picked
    e = prod.abs().sum(2) * ((D / 32 + 22) * ref.U32)
    want = prod.sum(2)
    ref.check(alone, want.cpu(), (e + ref.rounding(want.abs() + e, F32)).cpu(), "dweight")
