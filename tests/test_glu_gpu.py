"""GPU parity of the gated linear layer (glu_forward, glu_backward) against
its 64-bit definition: every tile path, types, activations, bias, stored
pre-activations, strides and alignments, the empty problems, accumulation,
in-place dP, capture, and what lies outside the matrices."""
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
CANARY = 321.0


@pytest.fixture(scope="module")
def g():
    import mixed_precision_dense_sm_gb300 as lib
    h = lib.Gemm()
    yield h
    h.close()


def matrix(rows, cols, dtype, gen, scale=1.0, pad=0, off=0):
    """A rows x cols CUDA view with `pad` further columns and `off` elements
    before it, all of which hold a canary."""
    buf = torch.full((rows * (cols + pad) + off + 8,), CANARY, dtype=dtype)
    v = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if gen is not None:
        v.copy_((torch.randn(rows, cols, generator=gen) * scale).to(dtype))
    dev = buf.cuda()
    return dev[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], dev


def around_intact(view, buf):
    rows, cols = view.shape
    mark = torch.zeros(buf.shape, dtype=torch.bool, device=buf.device)
    at = view.storage_offset()
    if rows:
        mark[at:at + rows * view.stride(0)].view(rows, -1)[:, :cols] = True
    return bool((buf[~mark] == CANARY).all())


def forward_case(g, M, F, K, dt, act, ht=None, bias=None, save=True, pad=(0, 0, 0, 0), off=(0, 0, 0, 0),
                 seed=0):
    ht = ht or dt
    gen = torch.Generator().manual_seed(seed + M + 3 * F + 7 * K)
    X, _ = matrix(M, K, dt, gen, pad=pad[0], off=off[0])
    W, _ = matrix(2 * F, K, dt, gen, scale=max(K, 1) ** -0.5, pad=pad[1], off=off[1])
    b = None if bias is None else torch.randn(2 * F, generator=gen).to(bias).cuda()
    H, hb = matrix(M, F, ht, None, pad=pad[2], off=off[2])
    P, pb = matrix(M, 2 * F, ht, None, pad=pad[3], off=off[3]) if save else (None, None)
    g.glu(X, W, H, act=act, bias=b, P=P)
    g.sync()
    rH, tH, rP, tP = ref.glu_forward(X.cpu(), W.cpu(), act, None if b is None else b.cpu(), ht)
    ref.check(H, rH, tH, "H")
    assert around_intact(H, hb)
    if save:
        ref.check(P, rP, tP, "P")
        assert around_intact(P, pb)
    return X, W, b, H, P


# one token to a large batch, both sides of every tile boundary, odd sizes
SHAPES = [(1, 64, 64), (1, 512, 1024), (2, 129, 200), (7, 1000, 333), (16, 640, 512), (33, 96, 4096),
          (64, 1024, 512), (65, 1024, 512), (100, 2176, 2048), (128, 64, 320), (129, 257, 129),
          (200, 31, 77), (255, 63, 64), (256, 4096, 256), (300, 1023, 777), (513, 128, 2112),
          (700, 1500, 136), (1000, 2048, 640), (1, 1, 1), (3, 8, 8), (40, 65, 72)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_forward_shapes(g, shape, dt):
    forward_case(g, *shape, dt, "silu" if dt is BF else "gelu", save=shape[0] % 2 == 0,
                 bias=F32 if shape[1] % 2 == 0 else None)


@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
@pytest.mark.parametrize("M", [5, 300, 2000])
def test_forward_activations_and_types(g, act, M):
    forward_case(g, M, 520, 192, BF, act, bias=BF)
    forward_case(g, M, 520, 192, FP, act, ht=F32, bias=FP)
    forward_case(g, M, 520, 192, BF, act, ht=FP, bias=F32)


@pytest.mark.parametrize("M", [9, 260, 1500])
@pytest.mark.parametrize("pad,off", [((8, 8, 8, 8), (0, 0, 0, 0)), ((1, 3, 5, 7), (0, 0, 0, 0)),
                                     ((0, 0, 0, 0), (1, 1, 1, 1)), ((0, 0, 4, 4), (8, 8, 4, 4))])
def test_forward_strides(g, M, pad, off):
    forward_case(g, M, 264, 256, BF, "silu", bias=F32, pad=pad, off=off)


def test_forward_large_pair_tiles(g):
    """CTA-pair tiles with several tiles per pair (TMA stores of H and P)."""
    forward_case(g, 2304, 4200, 128, BF, "silu", bias=F32)
    forward_case(g, 2048, 4096, 192, FP, "gelu", save=False)
    forward_case(g, 1030, 8200, 64, BF, "relu", ht=F32)


def test_forward_special_values(g):
    """Infinities and NaN follow act(g) * u; a large negative gate gives 0."""
    X = torch.zeros(4, 64, dtype=BF)
    X[0, 0], X[1, 0], X[2, 0], X[3, 0] = float("inf"), float("nan"), -2000.0, 2000.0
    W = torch.zeros(16, 64, dtype=BF)
    W[:, 0] = 1.0
    H = g.glu(X.cuda(), W.cuda(), act="silu").float().cpu()
    assert torch.isinf(H[0]).all() and torch.isnan(H[1]).all()
    assert (H[2].abs() == 0).all() and torch.allclose(H[3], torch.full((8,), 4e6), rtol=1e-2)


def test_forward_empty(g):
    X, W = torch.randn(0, 64, device="cuda").to(BF), torch.randn(32, 64, device="cuda").to(BF)
    assert g.glu(X, W).shape == (0, 16)
    assert g.glu(torch.randn(5, 64, device="cuda").to(BF), W[:0]).shape == (5, 0)
    b = torch.randn(32, device="cuda")
    H, P = torch.empty(5, 16, dtype=F32, device="cuda"), torch.empty(5, 32, dtype=F32, device="cuda")
    g.glu(torch.empty(5, 0, dtype=BF, device="cuda"), torch.empty(32, 0, dtype=BF, device="cuda"), H,
          bias=b, P=P)
    assert torch.equal(P, b.expand(5, 32))
    want = torch.nn.functional.silu(b[:16].double()) * b[16:].double()
    ref.check(H, want.cpu().expand(5, 16), 1e-5 * want.abs().cpu() + 1e-7, "K = 0")


def test_forward_repeats_bit_for_bit(g):
    X, W, b, H, P = forward_case(g, 64, 2048, 4096, FP, "silu", bias=F32)
    for _ in range(3):
        assert torch.equal(g.glu(X, W, bias=b), H)


def backward_case(g, M, F, K, dt, act, pt=None, dxt=None, dwt=None, beta_w=0.0, bias=F32, pad=0, off=0,
                  in_place=False, seed=0):
    pt, dxt, dwt = pt or dt, dxt or dt, dwt or dt
    gen = torch.Generator().manual_seed(seed + M + 3 * F + 7 * K)
    X, _ = matrix(M, K, dt, gen, pad=pad, off=off)
    W, _ = matrix(2 * F, K, dt, gen, scale=max(K, 1) ** -0.5, pad=pad, off=off)
    P, pb = matrix(M, 2 * F, pt, gen, pad=pad, off=off)
    dH, _ = matrix(M, F, dt, gen, scale=0.1, pad=pad, off=off)
    dP, dpb = (P, pb) if in_place else matrix(M, 2 * F, dt, None, pad=pad, off=off)
    dX, dxb = matrix(M, K, dxt, None, pad=pad, off=off)
    dW, dwb = matrix(2 * F, K, dwt, gen if beta_w else None, pad=pad, off=off)
    db = torch.empty(2 * F, dtype=bias, device="cuda") if bias is not None else None
    P0, dW0 = P.cpu(), dW.cpu()
    g.glu_backward(dH, P, X, W, act=act, dP=dP, dX=dX, dW=dW, dbias=db, beta_w=beta_w)
    g.sync()
    want = ref.glu_backward(dH.cpu(), P0, X.cpu(), W.cpu(), act, dt, dxt, dwt, beta_w, dW0)
    ref.check(dP, *want["dP"], "dP")
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW"], "dW")
    if db is not None:
        r, t = want["dbias"]
        ref.check(db, r, t + ref.rounding(r.abs() + t, bias), "dbias")
    assert around_intact(dP, dpb) and around_intact(dX, dxb) and around_intact(dW, dwb)


@pytest.mark.parametrize("shape", [(1, 64, 64), (2, 129, 200), (7, 1000, 333), (64, 1024, 512),
                                   (129, 257, 129), (300, 1023, 777), (513, 128, 2112), (1000, 2048, 640),
                                   (1, 1, 1), (40, 65, 72), (2100, 300, 264)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward_shapes(g, shape):
    backward_case(g, *shape, BF, "silu")
    backward_case(g, *shape, FP, "gelu", bias=None)


@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
def test_backward_types(g, act):
    backward_case(g, 150, 264, 136, BF, act, pt=F32, dxt=F32, dwt=F32, bias=BF)
    backward_case(g, 150, 264, 136, FP, act, pt=BF, dxt=BF, dwt=FP, bias=FP)


def test_backward_accumulates(g):
    backward_case(g, 200, 264, 136, BF, "silu", dwt=F32, beta_w=1.0)
    backward_case(g, 200, 264, 136, BF, "silu", beta_w=0.5)


def test_backward_in_place_and_strides(g):
    backward_case(g, 333, 264, 136, BF, "gelu", in_place=True)
    backward_case(g, 333, 263, 136, BF, "gelu", in_place=True, pad=3)
    backward_case(g, 333, 264, 136, BF, "gelu", pad=8, off=8)
    backward_case(g, 333, 264, 136, FP, "gelu", off=1)


def test_backward_without_products_and_empty(g):
    dH, P = torch.randn(4, 8, device="cuda").to(BF), torch.randn(4, 16, device="cuda").to(BF)
    dP = g.glu_backward(dH, P, None, None, act="relu")
    w = ref.glu_backward(dH.cpu(), P.cpu(), None, None, "relu", BF, BF, BF)["dP"]
    ref.check(dP, *w, "dP")
    dW, db = torch.ones(16, 24, device="cuda"), torch.ones(16, device="cuda")
    X0, W = torch.empty(0, 24, dtype=BF, device="cuda"), torch.randn(16, 24, device="cuda").to(BF)
    g.glu_backward(dH[:0], P[:0], X0, W, dX=torch.empty_like(X0), dW=dW, dbias=db, beta_w=0.5)
    assert (dW == 0.5).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["gelu", "silu", None])
def test_backward_against_differences(g, act):
    """The gradient of sum(H * R) by central differences of the 64-bit forward
    pass, at the same points: 2^-8 of the largest entry covers dP's and the
    result's bf16 roundings, with a step's own error below 1e-6."""
    gen = torch.Generator().manual_seed(3)
    M, F, K = 6, 16, 32
    X = torch.randn(M, K, generator=gen).to(BF)
    W = (torch.randn(2 * F, K, generator=gen) * K ** -0.5).to(BF)
    R = torch.randn(M, F, generator=gen).to(BF)
    P = torch.empty(M, 2 * F, dtype=F32, device="cuda")
    g.glu(X.cuda(), W.cuda(), torch.empty(M, F, dtype=F32, device="cuda"), act=act, P=P)
    dX = torch.empty(M, K, dtype=F32, device="cuda")
    dW = torch.empty(2 * F, K, dtype=F32, device="cuda")
    g.glu_backward(R.cuda(), P, X.cuda(), W.cuda(), act=act, dX=dX, dW=dW)

    def loss(x, w):
        p = x @ w.t()
        return (ref.act64(act, p[:, :F])[0] * p[:, F:] * R.double()).sum()
    h = 1e-5
    for got, base, which in ((dX, X, 0), (dW, W, 1)):
        num = torch.zeros(base.shape, dtype=torch.float64)
        for i in range(base.numel()):
            d = torch.zeros(base.numel(), dtype=torch.float64)
            d[i] = h
            d = d.view(base.shape)
            args = [X.double(), W.double()]
            hi, lo = list(args), list(args)
            hi[which] = args[which] + d
            lo[which] = args[which] - d
            num.view(-1)[i] = (loss(*hi) - loss(*lo)) / (2 * h)
        assert (got.cpu().double() - num).abs().max() <= 2.0 ** -8 * num.abs().max()


def test_capture_replays_with_new_inputs(g):
    """Forward and backward in one graph, on a side stream; replayed on other inputs."""
    M, F, K = 64, 1024, 1536
    gen = torch.Generator().manual_seed(5)
    X = torch.randn(M, K, generator=gen).to(BF).cuda()
    W = (torch.randn(2 * F, K, generator=gen) * K ** -0.5).to(BF).cuda()
    dH = torch.randn(M, F, generator=gen).to(BF).cuda()
    H, P = torch.empty(M, F, dtype=BF, device="cuda"), torch.empty(M, 2 * F, dtype=BF, device="cuda")
    dP, dX, dW = torch.empty_like(P), torch.empty_like(X), torch.empty_like(W)

    def step():
        g.glu(X, W, H, P=P)
        g.glu_backward(dH, P, X, W, dP=dP, dX=dX, dW=dW)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # a larger call outgrows the workspace that the graph uses
    big = torch.randn(512, 1001, device="cuda").to(BF)
    g.glu(big, torch.randn(2 * 3001, 1001, device="cuda").to(BF))
    X.copy_(torch.randn(M, K, generator=gen).to(BF))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (H, P, dP, dX, dW)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (H, P, dP, dX, dW)))


@pytest.mark.parametrize("mode", ["global", "thread_local", "relaxed"])
def test_capture_grows_the_workspace(mode):
    """First calls of a handle under capture, each with more workspace than the
    last; the graph stays right once larger calls have outgrown its buffers."""
    import mixed_precision_dense_sm_gb300 as lib
    h = lib.Gemm()
    gen = torch.Generator().manual_seed(6)
    Xs = [torch.randn(M, 1001, generator=gen).to(BF).cuda() for M in (30, 300, 600)]
    W = (torch.randn(600, 1001, generator=gen) / 32).to(BF).cuda()
    Hs = [torch.empty(X.shape[0], 300, dtype=BF, device="cuda") for X in Xs]
    C = torch.empty(300, 600, dtype=BF, device="cuda")

    def step():
        for X, H in zip(Xs, Hs):
            h.glu(X, W, H)                       # unaligned rows: copied to the workspace
        h(Xs[1], W, C, transB="T")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode=mode):
        step()
    h.glu(torch.cat(Xs * 4), W)                  # outgrows it again
    for t in (*Hs, C):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*Hs, C)]
    other = lib.Gemm()
    h, mine = other, h
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (*Hs, C)))
    del graph
    mine.close()
    other.close()


@pytest.mark.parametrize("shape", [(300, 256, 512), (16, 640, 1024), (64, 20480, 256), (2048, 2048, 256)],
                         ids=lambda s: "x".join(map(str, s)))
def test_a_load_that_never_lands_is_reported(shape):
    """The planted missing load (gemm_debug_set) on each tile path: the wait
    runs out, the kernel winds down, the handle reports it and works again."""
    import mixed_precision_dense_sm_gb300 as lib
    h = lib.Gemm()
    M, F, K = shape
    X, W = torch.randn(M, K, device="cuda").to(BF), torch.randn(2 * F, K, device="cuda").to(BF)
    want = h.glu(X, W)
    h.sync()
    assert lib.gemm_debug_set(h.h, lib.GEMM_DEBUG_SKIP_FIRST_LOAD, 20_000_000) == 0
    h.glu(X, W)
    with pytest.raises(lib.GemmError) as e:
        h.sync()
    assert e.value.status == 5
    assert lib.gemm_debug_set(h.h, 0, 0) == 0
    got = h.glu(X, W)
    h.sync()
    assert torch.equal(got, want)
    h.close()


# tokens around the few-token kernels' bounds, splits of K over 1 to 8 CTAs,
# more tiles than two per SM
@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("F,K", [(64, 2048), (100, 520), (1024, 1024), (4100, 640), (20480, 128), (200, 4096)])
def test_forward_few_tokens(g, M, F, K):
    forward_case(g, M, F, K, FP, "gelu", bias=F32, save=M % 2 == 1)


@pytest.mark.parametrize("M", [1, 2])
def test_rows_of_almost_2_to_the_31(g, M):
    """A few tokens of the longest rows: zeros but for the first and the last
    elements, whose products are exact."""
    K, F = 2 ** 31 - 8, 1
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    X, W = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(2 * F, K, dtype=BF, device="cuda")
    for t in (X, W):
        t[:, :8] = 2
        t[:, -8:] = torch.arange(1, 9, device="cuda").to(BF)
    W[1] *= -1
    H = g.glu(X, W, act="none")
    P = 8 * 4 + sum(i * i for i in range(1, 9))            # 236
    assert (H.float() == torch.tensor(-P * P, dtype=torch.float32).to(BF).float()).all()
    del X, W
    torch.cuda.empty_cache()


def test_refusals_on_the_device(g):
    import mixed_precision_dense_sm_gb300 as lib
    X, W = torch.randn(8, 32, device="cuda").to(BF), torch.randn(16, 32, device="cuda").to(BF)
    for bad in (lambda: g.glu(X, W[:15]), lambda: g.glu(X.t(), W), lambda: g.glu(X, W.half()),
                lambda: g.glu(X.cpu(), W), lambda: g.glu(X, W, bias=torch.ones(8, device="cuda")),
                lambda: g.glu(X, W, P=torch.empty(8, 16, dtype=FP, device="cuda")),
                lambda: g.glu_backward(X, torch.empty(8, 60, dtype=BF, device="cuda"), X, W)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.GemmError) as e:
        g.glu(X.float(), W.float())
    assert e.value.status == 2
