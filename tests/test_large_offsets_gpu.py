"""Matrices and tensors of more than 2^31 elements: what lies behind an offset
of 32 bits is read and written like the rest."""
import math

import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    yield lib
    torch.cuda.empty_cache()


def need(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def filled(M, N, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(M, N, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // N)
    for i in range(0, M, step):
        part = t[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return t


@pytest.mark.parametrize("N,kind", [(8192, "rms"), (4095, "layer"), (12288, "layer")])
def test_norm_rows(lib, N, kind):
    """Rows are independent: the last ones of a long call are those of a short one."""
    need(80)
    M, tail = 2 ** 31 // N + 1500, 700
    X, Z, dY = (filled(M, N, BF, s) for s in (1, 2, 3))
    w = torch.rand(N, device="cuda") + 0.5
    kw = dict(pre=kind, pre_weight=w, post=kind, post_weight=w)
    XO, Y = lib.norm_block(X, Z, **kw)
    a, b = lib.norm_block(X[-tail:], Z[-tail:], **kw)
    assert torch.equal(XO[-tail:], a) and torch.equal(Y[-tail:], b)
    a, b = lib.norm_block(X[:tail], Z[:tail], **kw)
    assert torch.equal(XO[:tail], a) and torch.equal(Y[:tail], b)
    del Y
    dX, dZ, dw, db = torch.empty_like(X), torch.empty_like(Z), torch.empty_like(w), torch.empty_like(w)
    lib.norm_block_backward(XO, dY, X, Z, dX=dX, dZ=dZ, dpre_weight=dw, dpre_bias=db, **kw)
    for part in (slice(M - tail, M), slice(0, tail)):
        a, b = torch.empty(tail, N, dtype=BF, device="cuda"), torch.empty(tail, N, dtype=BF, device="cuda")
        lib.norm_block_backward(XO[part], dY[part], X[part], Z[part], dX=a, dZ=b, dpre_weight=dw.clone(),
                                dpre_bias=dw.clone(), **kw)
        assert torch.equal(dX[part], a) and torch.equal(dZ[part], b)
    # a column's sum in 64 bits, at the tolerance of FP32 sums of M values
    for c in (0, N - 1):
        col = dY[:, c].double()
        assert abs(float(db[c]) - float(col.sum())) <= (M + 64) * ref.U32 * float(col.abs().sum())


@pytest.mark.parametrize("K,F", [(256, 8192), (264, 8191)])
def test_gated_layer_rows(lib, K, F):
    need(120)
    g = lib.Gemm()
    M, tail = 2 ** 31 // (2 * F) + 3000, 2000            # (P's rows pass 2^31 elements)
    X = filled(M, K, BF, 4)
    W = filled(2 * F, K, BF, 5, scale=K ** -0.5)
    P = torch.empty(M, 2 * F, dtype=BF, device="cuda")
    H = g.glu(X, W, act="silu", P=P)
    g.sync()
    rows = torch.tensor([0, 1, M // 2, M - 130, M - 2, M - 1])
    h, eh, p, ep = ref.glu_forward(X[rows.cuda()].cpu(), W.cpu(), "silu", None, BF)
    ref.check(H[rows.cuda()], h, eh, "H")
    ref.check(P[rows.cuda()], p, ep, "P")
    dW = torch.empty(2 * F, K, dtype=F32, device="cuda")
    dX = torch.empty_like(X)
    kept = P[rows.cuda()].cpu()
    dH = H
    dh = dH[rows.cuda()].cpu()
    g.glu_backward(dH, P, X, W, dP=P, dX=dX, dW=dW)
    g.sync()
    want = ref.glu_backward(dh, kept, X[rows.cuda()].cpu(), W.cpu(), "silu", BF, BF, F32)
    ref.check(P[rows.cuda()], *want["dP"], "dP")
    ref.check(dX[rows.cuda()], *want["dX"], "dX")
    # A row of dW from dP as stored.  One step of the tensor core adds 16 products
    # to the sum and cuts each of the 17 terms below 2^-23 of the largest, so M
    # products are off by at most M / 16 * 17 * 2^-23 times the largest sum on the way.
    for f in (0, 2 * F - 1):
        prod = P[:, f, None].double() * X[:, :4].double()
        most = prod.cumsum(0).abs().amax(0) + prod.abs().amax(0)
        assert ((dW[f, :4].double() - prod.sum(0)).abs() <= M / 16 * 17 * 2.0 ** -23 * most).all()
    # and where all but a few rows give no gradient: as many products in each sum
    dH = torch.zeros_like(H)
    dH[rows.cuda()] = dh.cuda()
    P[rows.cuda()] = kept.cuda()
    g.glu_backward(dH, P, X, W, dP=P, dW=dW)
    g.sync()
    ref.check(dW, *ref.glu_backward(dh, kept, X[rows.cuda()].cpu(), None, "silu", BF, BF, F32)["dW"], "dW")
    g.close()


@pytest.mark.parametrize("dt,off", [(BF, 0), (FP, 1)], ids=["bf16", "fp16_unaligned"])
def test_clipping_one_large_tensor(lib, dt, off):
    need(60)
    n = 2 ** 32 + 12345
    g = torch.zeros(n + off, dtype=dt, device="cuda")[off:]
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 7, n - 1], device="cuda")
    v = torch.tensor([1.0, 2.0, 2.0, 4.0, 4.0, 8.0], device="cuda", dtype=dt)
    g[at] = v
    out = torch.ones(n, dtype=dt, device="cuda")
    norm = math.sqrt(float(v.double().square().sum()))
    got = lib.grad_clip([g], 1.0, outputs=[out])
    assert abs(float(got) - norm) <= 8 * ref.U32 * norm
    r = v.cpu().double() / norm
    ref.check(out[at], r, 11 * ref.U32 * r + ref.rounding(r, dt), "out")
    assert int(torch.count_nonzero(out)) == 6
