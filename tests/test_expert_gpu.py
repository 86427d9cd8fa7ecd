"""GPU parity of the experts' row moves against their definitions in 64 bits
(expert_ref): sizes from one token on, dropped choices, types, weights, pitches and
alignments, more choices than a turn, special values, streams, capture."""
import pytest
import torch

import expert_ref as ex
import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16", F32: "fp32"}


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def choices(T, k, E, drop=0.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=gen)
    ids[torch.rand(T, k, generator=gen) < drop] = -1
    return ids


def pitched(rows, cols, dtype, pad, off=0, fill=77.0, gen=None):
    """A matrix of pitch cols + pad that starts `off` elements into its memory."""
    buf = torch.full((off + rows * (cols + pad),), fill, dtype=dtype, device="cuda")
    m = buf[off:].view(rows, cols + pad)[:, :cols]
    if gen is not None:
        m.copy_(torch.randn(rows, cols, generator=gen).to(dtype))
    return m, buf


# ------------------------------------------------------------------------- sort

def check_sort(lib, ids, E, dtype, pitch=0):
    T, k = ids.shape
    dev = torch.full((T, k + pitch), -5, dtype=dtype, device="cuda")
    dev[:, :k] = ids.to(dtype)
    got = lib.expert_sort(dev[:, :k], E)
    for g, r, n in zip(got, ex.sort(ids, E), ("pos", "offsets", "order")):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), r), n


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", [(0, 4, 3), (5, 0, 3), (1, 1, 1), (1, 8, 64), (31, 1, 7), (33, 3, 1024),
                                   (64, 8, 128), (1000, 3, 33), (4096, 1, 16), (4097, 1, 31), (8192, 8, 128),
                                   (5000, 7, 999), (40000, 5, 60)])
def test_sort(lib, T, k, E, dtype):
    check_sort(lib, choices(T, k, E, seed=T + k), E, dtype)
    check_sort(lib, choices(T, k, E, drop=0.4, seed=T), E, dtype, pitch=3)


@pytest.mark.parametrize("T,k,E", [(131072, 1, 9), (131073, 1, 1024), (135167, 1, 500), (33792, 4, 64), (70000, 3, 2),
                                   (2 ** 20, 8, 1024)])
def test_sort_of_many_slots(lib, T, k, E):
    """Around the border of the one-launch form and of its last CTA's share, against
    torch's stable sort."""
    for drop, dtype in ((0.0, torch.int64), (0.5, torch.int32)):
        ids = choices(T, k, E, drop, seed=E)
        if drop:
            ids[:: 7] = E - 1
        pos, offsets, order = (t.cpu().long() for t in lib.expert_sort(ids.to(dtype).cuda(), E))
        key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
        kept = int((key < E).sum())
        want = torch.sort(key, stable=True)[1]
        want[kept:] = -1
        assert torch.equal(order, want)
        counts = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
        assert torch.equal(offsets, torch.cat([torch.zeros(1, dtype=torch.int64), counts]))
        back = torch.full((T * k,), -1)
        back[order[:kept]] = torch.arange(kept)
        assert torch.equal(pos.flatten(), back)


@pytest.mark.parametrize("T,k,E", [(3000, 2, 50), (30000, 6, 300), (140000, 1, 700)])
def test_sort_extremes(lib, T, k, E):
    """All choices one expert's, the last expert's, none at all, ids at the types' ends."""
    for v in (0, E - 1, E, -1, 2 ** 31 - 1, -2 ** 31):
        check_sort(lib, torch.full((T, k), v), E, torch.int32)
    for v in (2 ** 40, -2 ** 40, 2 ** 32, 2 ** 63 - 1):
        check_sort(lib, torch.full((T, k), v), E, torch.int64)


def test_sort_into_given_tensors(lib):
    ids = choices(100, 4, 9)
    pos, offsets, order = (torch.full(s, 5, dtype=torch.int32, device="cuda") for s in ((100, 4), (10,), (400,)))
    got = lib.expert_sort(ids.cuda(), 9, pos, offsets, order)
    assert got[0] is pos and got[1] is offsets and got[2] is order
    assert torch.equal(order.cpu(), ex.sort(ids, 9)[2])
    st = lib.expert_sort_raw(100, 4, 9, ids.cuda().data_ptr(), 4, 8, pos.zero_().data_ptr(), offsets.data_ptr(),
                             0, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(pos.cpu(), ex.sort(ids, 9)[0])


# ------------------------------------------------------------------------- rows

def problem(T, k, D, dtype, wtype, drop, pad=0, off=0, E=5, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * D + T)
    pos = ex.sort(choices(T, k, E, drop, seed), E)[0]
    x, _ = pitched(T, D, dtype, pad, off, gen=gen)
    rows, _ = pitched(T * k, D, dtype, pad, off, gen=gen)
    w = None
    if wtype is not None:
        w = pitched(T, k, wtype, 1 if pad else 0, gen=gen)[0]
    return pos, x, rows, w


def cpu(t):
    return None if t is None else t.cpu()


def check_rows(lib, pos, x, rows, w, pad=0, off=0, dw_type=None):
    T, k = pos.shape
    D, dt = x.shape[1], x.dtype
    p = pos.cuda()
    before, buf = pitched(T * k, D, dt, pad, off)
    hull = buf.clone()
    lib.expert_gather(x, p, w, Xs=before)
    r, tol = ex.out(x.cpu(), pos, cpu(w), torch.full((T * k, D), 77.0, dtype=dt))
    ref.check(before, r, tol, "Xs")
    before.fill_(77.0)
    assert torch.equal(buf, hull), "padding"

    y, buf = pitched(T, D, dt, pad, off)
    hull = buf.clone()
    lib.expert_combine(rows, p, w, Y=y)
    r, tol = ex.back(rows.cpu(), pos, cpu(w), D)
    ref.check(y, r, tol, "Y")
    y.fill_(77.0)
    assert torch.equal(buf, hull), "padding"

    dwt = dw_type or (w.dtype if w is not None else F32)
    dx, dw = torch.empty(T, D, dtype=dt, device="cuda"), torch.empty(T, k, dtype=dwt, device="cuda")
    lib.expert_gather_backward(rows, p, w, x, dX=dx, dweight=dw)
    ref.check(dx, r, tol, "dX")
    d, dtol = ex.dots(x.cpu(), rows.cpu(), pos, dwt)
    ref.check(dw, d, dtol, "dweight")
    if D:
        only = torch.empty_like(dw)
        lib.expert_gather_backward(rows, p, w, x, dweight=only)
        # (not the same bits: without dX the rows may be vectors, which is another order)
        ref.check(only, d, dtol, "dweight alone")

    r, tol = ex.out(x.cpu(), pos, cpu(w), torch.full((T * k, D), 77.0, dtype=dt))
    dys = torch.full((T * k, D), 77.0, dtype=dt, device="cuda")
    lib.expert_combine_backward(x, p, w, rows, dYs=dys, dweight=dw.zero_())
    ref.check(dys, r, tol, "dYs")
    ref.check(dw, d, dtol, "dweight")
    # in place over Ys, and without the weights' gradient
    inplace = rows.clone()
    lib.expert_combine_backward(x, p, w, inplace, dYs=inplace, dweight=dw.zero_())
    ref.check(dw, d, dtol, "dweight in place")
    named = pos[pos >= 0].long()
    assert torch.equal(inplace[named.cuda()], dys[named.cuda()])
    lib.expert_combine_backward(x, p, w, dYs=inplace.fill_(77.0))
    assert torch.equal(inplace, dys)


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=IDS.get)
@pytest.mark.parametrize("T,k,D", [(1, 1, 1), (1, 8, 4096), (2, 3, 7), (5, 2, 8), (64, 8, 64), (7, 4, 1000),
                                   (33, 9, 130), (3, 17, 520), (400, 2, 136), (10, 3, 5000), (700, 1, 24),
                                   (4, 2, 2055), (6, 3, 1027)])
def test_rows(lib, T, k, D, dtype):
    check_rows(lib, *problem(T, k, D, dtype, F32, 0.0))
    check_rows(lib, *problem(T, k, D, dtype, None, 0.3, seed=1))


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=IDS.get)
@pytest.mark.parametrize("T,k,D", [(10000, 3, 256), (9777, 7, 320), (1300, 8, 2048), (1250, 2, 5000), (12000, 1, 264),
                                   (1400, 4, 4104)])
def test_many_tokens(lib, T, k, D, dtype):
    """Enough tokens for the ring, against 64 bits on the GPU: the same bounds."""
    pos, x, rows, w = problem(T, k, D, dtype, F32, 0.2)
    p, on = pos.cuda(), (pos >= 0).cuda()
    X, R, W = x.double(), rows.double(), torch.where(on, w.double(), 0.0)
    at = p.long().clamp(min=0)
    y, mag = torch.zeros_like(X), torch.zeros_like(X)
    d, dmag = torch.zeros_like(W), torch.zeros_like(W)
    for j in range(k):
        r = R[at[:, j]] * on[:, j : j + 1]
        y += r * W[:, j : j + 1]
        mag += (r * W[:, j : j + 1]).abs()
        d[:, j], dmag[:, j] = (X * r).sum(1), (X * r).abs().sum(1)
    e = mag * (k * ref.U32)
    tol = e + ref.rounding(y.abs() + e, dtype)
    de = dmag * ((D / 32 + 22) * ref.U32)
    dtol = de + ref.rounding(d.abs() + de, F32)
    ref.check(lib.expert_combine(rows, p, w), y.cpu(), tol.cpu(), "Y")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    lib.expert_gather_backward(rows, p, w, x, dX=dx, dweight=dw)
    ref.check(dx, y.cpu(), tol.cpu(), "dX")
    ref.check(dw, d.cpu(), dtol.cpu(), "dweight")
    out, otol = torch.full_like(R, 77.0), torch.zeros_like(R)
    t, j = torch.nonzero(on, as_tuple=True)
    v = X[t] * W[t, j][:, None]
    out[at[t, j]] = v
    otol[at[t, j]] = v.abs() * ref.U32 + ref.rounding(v.abs() * (1 + ref.U32), dtype)
    got = torch.full_like(rows, 77.0)
    lib.expert_combine_backward(x, p, w, rows, dYs=got, dweight=dw.zero_())
    ref.check(got, out.cpu(), otol.cpu(), "dYs")
    ref.check(dw, d.cpu(), dtol.cpu(), "dweight")
    ref.check(lib.expert_gather(x, p, w, Xs=got.fill_(77.0)), out.cpu(), otol.cpu(), "Xs")
    lib.expert_combine_backward(x, p, w, rows, dYs=rows, dweight=dw.zero_())
    ref.check(dw, d.cpu(), dtol.cpu(), "dweight in place")
    assert torch.equal(rows[at[t, j]], got[at[t, j]])


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=IDS.get)
@pytest.mark.parametrize("pad,off", [(8, 0), (1, 0), (0, 1), (4, 3), (16, 8)])
def test_pitches_and_alignment(lib, dtype, pad, off):
    for T, k, D in ((9, 3, 77), (40, 5, 264), (350, 2, 1023)):
        check_rows(lib, *problem(T, k, D, dtype, dtype, 0.2, pad, off), pad=pad, off=off)


@pytest.mark.parametrize("wtype", [BF, FP, F32], ids=IDS.get)
def test_weight_types(lib, wtype):
    for dwt in (BF, FP, F32):
        check_rows(lib, *problem(30, 4, 96, BF, wtype, 0.1), dw_type=dwt)


def test_empty(lib):
    for T, k, D in ((0, 2, 8), (3, 0, 8), (3, 2, 0)):
        check_rows(lib, *problem(T, k, D, BF, F32, 0.0))


def test_all_dropped_and_outside(lib):
    """Tokens without choices get zeros whatever the rows hold; positions that are
    no rows count as none."""
    pos = torch.tensor([[-1, -1], [0, 9], [-7, 2 ** 31 - 1]], dtype=torch.int32)
    rows = torch.full((4, 24), float("nan"), device="cuda")
    rows[0] = 2.0
    w = torch.full((3, 2), 3.0, device="cuda")
    y = lib.expert_combine(rows, pos.cuda(), w)
    assert torch.equal(y.cpu(), torch.tensor([0.0, 6.0, 0.0])[:, None].expand(3, 24))
    dw = torch.full((3, 2), 5.0, device="cuda")
    lib.expert_gather_backward(rows, pos.cuda(), w, torch.ones(3, 24, device="cuda"), dweight=dw)
    assert torch.equal(dw.cpu(), torch.tensor([[0.0, 0.0], [48.0, 0.0], [0.0, 0.0]]))
    xs = lib.expert_gather(torch.ones(3, 24, device="cuda"), pos.cuda(), Xs=rows.fill_(7.0))
    assert torch.equal(xs.cpu(), torch.tensor([1.0, 7.0, 7.0, 7.0])[:, None].expand(4, 24))


@pytest.mark.parametrize("D", [16, 77])
def test_special_values(lib, D):
    """Infinities and NaN where IEEE arithmetic has them, overflow included."""
    pos = torch.arange(8, dtype=torch.int32).view(4, 2)
    x = torch.ones(4, D, dtype=FP)
    x[0, 3], x[1, 5], x[2, 7], x[3] = float("inf"), float("nan"), 65504.0, 60000.0
    w = torch.tensor([[0.0, 1.0], [1.0, 2.0], [2.0, -1.0], [float("inf"), float("nan")]])
    rows = torch.ones(8, D, dtype=FP)
    rows[2, 1], rows[5, 2] = float("-inf"), float("nan")
    xd, rd, wd = x.cuda(), rows.cuda(), w.cuda()
    want = (x.double()[:, None] * w.double()[..., None]).flatten(0, 1).float().half()
    assert torch.equal(lib.expert_gather(xd, pos.cuda(), wd).cpu().nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
    want = (rows.double().view(4, 2, D) * w.double()[..., None]).sum(1).float().half()
    assert torch.equal(lib.expert_combine(rd, pos.cuda(), wd).cpu().nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
    dw = torch.empty(4, 2, device="cuda")
    lib.expert_combine_backward(xd, pos.cuda(), wd, rd, dweight=dw)
    want = torch.einsum("td,tjd->tj", x.double(), rows.double().view(4, 2, D)).float()
    assert torch.equal(dw.cpu().isnan(), want.isnan()) and torch.equal(dw.cpu().isinf(), want.isinf())


def test_gradients_against_differences(lib):
    """Of f = sum(C * combine(gather(X, a), b)): linear in each factor, so a central
    difference is exact but for roundings: FP32 values of size about 1, sums of 12 * 40
    terms, a step of 1/2."""
    gen = torch.Generator().manual_seed(3)
    pos = ex.sort(choices(12, 3, 4, 0.2, 5), 4)[0].cuda()
    x, c = (torch.randn(12, 40, generator=gen).cuda() for _ in range(2))
    a, b = (torch.randn(12, 3, generator=gen).cuda() for _ in range(2))

    def f(x, a, b):
        xs = lib.expert_gather(x, pos, a, Xs=torch.zeros(36, 40, device="cuda"))
        return float((c.double() * lib.expert_combine(xs, pos, b).double()).sum())

    xs = lib.expert_gather(x, pos, a, Xs=torch.zeros(36, 40, device="cuda"))
    da, db, dx, dxs = torch.empty_like(a), torch.empty_like(b), torch.empty_like(x), torch.zeros_like(xs)
    lib.expert_combine_backward(c, pos, b, xs, dYs=dxs, dweight=db)
    lib.expert_gather_backward(dxs, pos, a, x, dX=dx, dweight=da)
    for arg, grad in ((0, dx), (1, da), (2, db)):
        for i in range(0, grad.numel(), 7):
            args = [x.clone(), a.clone(), b.clone()]
            args[arg].flatten()[i] += 0.5
            up = f(*args)
            args[arg].flatten()[i] -= 1.0
            diff = up - f(*args)
            # outputs of magnitude below 60 (4.5 sigma), two evaluations of 480 of them, 8 roundings each
            assert abs(diff - float(grad.flatten()[i])) <= 2 * 480 * 60 * 8 * ref.U32


def test_large_offsets(lib):
    """Rows behind 2^31 elements."""
    D, n = 2 ** 20, 2 ** 11 + 5
    rows = torch.empty(n, D, dtype=BF, device="cuda")
    pos = torch.tensor([[n - 1, 3], [2 ** 11 + 1, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, D, device="cuda").to(BF)
    lib.expert_gather(x, pos, Xs=rows)
    assert torch.equal(rows[n - 1], x[0]) and torch.equal(rows[3], x[0]) and torch.equal(rows[2 ** 11 + 1], x[1])
    y = lib.expert_combine(rows, pos)
    assert torch.equal(y[0], (2 * x[0].float()).to(BF)) and torch.equal(y[1], x[1])


def test_other_stream_and_capture(lib):
    ids = choices(200, 4, 16, 0.1)
    pos, x, rows, w = problem(200, 4, 128, BF, F32, 0.1, E=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids_d = ids.cuda()
    torch.cuda.synchronize()

    def chain():
        p, _, _ = lib.expert_sort(ids_d, 16)
        xs = lib.expert_gather(x, p, Xs=torch.zeros(800, 128, dtype=BF, device="cuda"))
        return p, lib.expert_combine(xs, p, w)

    want = chain()
    with torch.cuda.stream(s):
        got = chain()
    by_arg = lib.expert_combine(rows, pos.cuda(), w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    assert torch.equal(by_arg, lib.expert_combine(rows, pos.cuda(), w))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain()
    new = choices(200, 4, 16, 0.3, seed=9)
    ids_d.copy_(new)
    for _ in range(3):
        g.replay()
    want = chain()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals(lib):
    x, pos = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for bad in (lambda: lib.expert_sort(ids.float(), 4), lambda: lib.expert_sort(ids[0], 4),
                lambda: lib.expert_sort(ids.t(), 4), lambda: lib.expert_sort(ids, 4, pos=pos.long()),
                lambda: lib.expert_sort(ids, 4, offsets=torch.zeros(4, dtype=torch.int32, device="cuda")),
                lambda: lib.expert_gather(x, pos.long()), lambda: lib.expert_gather(x, pos[:3]),
                lambda: lib.expert_gather(x, pos.cpu()), lambda: lib.expert_gather(x.t(), pos),
                lambda: lib.expert_gather(x, pos, Xs=torch.zeros(8, 7, device="cuda")),
                lambda: lib.expert_gather(x, pos, Xs=torch.zeros(8, 8, device="cuda", dtype=BF)),
                lambda: lib.expert_gather(x, pos, torch.zeros(4, 3, device="cuda")),
                lambda: lib.expert_combine(x, pos, Y=torch.zeros(3, 8, device="cuda")),
                lambda: lib.expert_combine(x, torch.zeros(2, 4, dtype=torch.int32, device="cuda").t()),
                lambda: lib.expert_gather_backward(x, pos, dweight=torch.zeros(4, 2, device="cuda")),
                lambda: lib.expert_combine_backward(x, pos, dweight=torch.zeros(4, 2, device="cuda")),
                lambda: lib.expert_gather_backward(x, pos), lambda: lib.expert_combine_backward(x, pos)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.expert_sort(ids, 0, offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
                lambda: lib.expert_sort(ids, 1025),
                lambda: lib.expert_gather(x[:1].expand(4, 8), pos)):
        with pytest.raises(lib.GemmError) as e:
            bad()
        assert e.value.status == 1
