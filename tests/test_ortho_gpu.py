"""GPU parity of the orthogonalised update (ortho_update) against its definition in
64 bits (ortho_ref): sides from 1 on, both orientations, batches, types, pitches,
coefficients, magnitudes, special values, streams, capture, the wait that runs out."""
import pytest
import torch

import ortho_ref as ortho

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16", F32: "fp32"}


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


@pytest.fixture(scope="module")
def g(lib):
    h = lib.Gemm()
    yield h
    h.close()


def update(*shape, dtype=F32, seed=0, kind="noise", scale=1e-3):
    """A few strong directions over noise, noise alone, or a decaying spectrum."""
    gen = torch.Generator().manual_seed(seed + 3 * sum(shape))
    r, c = shape[-2:]
    n = torch.randn(*shape, generator=gen)
    if kind == "few":
        k = max(1, min(r, c) // 32)
        n = 0.3 * n + torch.randn(*shape[:-2], r, k, generator=gen) @ torch.randn(*shape[:-2], k, c, generator=gen)
    elif kind == "decay":
        k = min(r, c)
        u = torch.linalg.qr(torch.randn(r, k, generator=gen))[0]
        v = torch.linalg.qr(torch.randn(c, k, generator=gen))[0]
        n = (u * torch.logspace(0, -3, k)) @ v.T * k
    return (n * scale).to(dtype).cuda()


SHAPES = [(1, 1), (1, 100), (100, 1), (2, 3), (16, 16), (17, 70), (64, 64), (63, 65), (65, 63), (128, 128),
          (200, 130), (129, 512), (300, 700), (520, 257), (512, 2000)]


@pytest.mark.parametrize("kind", ["noise", "few", "decay"])
@pytest.mark.parametrize("r,c", SHAPES)
def test_shapes(g, r, c, kind):
    G = update(r, c, kind=kind)
    keep = G.clone()
    O = g.orthogonalize(G)
    g.sync()
    assert torch.equal(G, keep)
    ortho.check(O, G)


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=IDS.get)
@pytest.mark.parametrize("r,c", [(40, 300), (300, 40), (129, 133), (64, 256)])
def test_types_and_pitches(g, r, c, dtype):
    G = update(r, c, dtype=dtype, scale=1.0)
    ortho.check(g.orthogonalize(G), G)
    for pad, off in ((1, 0), (8, 0), (8, 1), (3, 5)):
        buf = torch.full((off + r * (c + pad),), 9.0, dtype=dtype, device="cuda")
        m = buf[off:].view(r, c + pad)[:, :c]
        m.copy_(G)
        out = torch.full((off + r * (c + pad),), 9.0, dtype=BF, device="cuda")
        o = out[off:].view(r, c + pad)[:, :c]
        hull = out.clone()
        g.orthogonalize(m, o)
        ortho.check(o, G)
        o.fill_(9.0)
        assert torch.equal(out, hull), "padding"


@pytest.mark.parametrize("batch,r,c", [(0, 8, 8), (1, 30, 50), (3, 64, 200), (5, 300, 200), (40, 33, 65), (9, 520, 640)])
def test_batches(g, batch, r, c):
    G = update(batch, r, c, kind="few", dtype=BF, scale=1.0)
    for i in range(batch):
        G[i] *= 2.0 ** (i - 2)
    O = g.orthogonalize(G)
    for i in range(batch):
        ortho.check(O[i], G[i])
    if batch > 1:
        # matrices that lie apart, every other one
        wide = torch.zeros(2 * batch, r, c + 8, dtype=BF, device="cuda")
        view = wide[::2, :, :c]
        got = g.orthogonalize(G, view)
        assert got is view and torch.equal(view, O)
        assert not wide[1::2].any() and not wide[:, :, c:].any()


def test_large_on_pairs(g):
    """Enough tiles for the CTA pairs' kernel in every product, odd sides."""
    G = update(2, 1500, 3000, kind="few", dtype=BF, scale=1.0)
    O = g.orthogonalize(G)
    T = g.orthogonalize(G.mT.contiguous())
    for i in range(2):
        want = ortho.define(G[i], (3.4445, -4.7750, 2.0315))
        near = ortho.rounded(G[i], (3.4445, -4.7750, 2.0315))
        # (the transposes have their sums in other orders)
        for got in (O[i].double(), T[i].mT.double()):
            # as measured on the sizes above, whose bound the singular values give: 2^-8 of the norm
            assert float((got - want).norm()) <= 2.0 ** -8 * float(want.norm())
            assert float((got - near).abs().max()) <= 2.0 ** -8 * float(near.abs().max())


def test_offsets_beyond_2_to_the_31(g):
    """The last of 34 matrices of 2^26 elements gives the bits that it gives alone."""
    G = torch.zeros(34, 8192, 8192, dtype=BF, device="cuda")
    G[33] = update(8192, 8192, dtype=BF, scale=1.0)
    G[0] = update(8192, 8192, dtype=BF, scale=0.5, seed=1)
    O = g.orthogonalize(G, steps=2)
    for i in (0, 33):
        assert torch.equal(O[i], g.orthogonalize(G[i], steps=2))
    assert not O[1:33].any() and bool(O[33].any())
    g.sync()


def test_coefficients_steps_and_scale(g):
    G = update(96, 160)
    for steps, abc in ((1, (1.5, -0.5, 0.0)), (8, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5)), (32, (1.5, -0.5, 0.0)),
                       (2, ((3.4, -4.7, 2.0), (1.9, -1.3, 0.4)))):
        for scale in (1.0, -0.25, 0.0):
            O = g.orthogonalize(G, steps=steps, coefficients=abc, scale=scale)
            ortho.check(O, G, abc, scale=scale, steps=steps)


def test_orthogonal_in_the_end(g):
    """Newton's own coefficients converge: rows with unit norms, at right angles,
    but for roundings to BF16 of 2^-9 each."""
    G = update(60, 256)
    O = g.orthogonalize(G, steps=24, coefficients=(1.5, -0.5, 0.0)).double()
    assert float((O @ O.mT - torch.eye(60, device="cuda")).abs().max()) <= 2 * 2.0 ** -9 * 1.01


@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1e-12, 1.0, 1e18, 1e34])
def test_magnitudes(g, scale):
    for r, c in ((24, 72), (72, 24)):
        G = update(r, c, scale=scale)
        ortho.check(g.orthogonalize(G, eps=0.0), G, eps=0.0)
        if scale >= 1e-12:
            ortho.check(g.orthogonalize(G), G)


def test_zeros_and_special_values(g):
    Z = torch.zeros(3, 40, 50, device="cuda")
    Z[1, 3, 4] = float("inf")
    Z[2] = update(40, 50)
    for G in (Z, Z.mT.contiguous()):
        O = g.orthogonalize(G)
        assert not O[0].any() and bool(O[1].isnan().all())
        ortho.check(O[2], G[2])
    G = update(70, 30)
    G[5, 6] = float("nan")
    assert bool(g.orthogonalize(G).isnan().all())
    # one element, one row, a row of one hot element
    one = torch.zeros(20, 90, device="cuda")
    one[7, 8] = -3.0
    ortho.check(g.orthogonalize(one), one)


def test_in_place_and_same_bits(g):
    G = update(130, 200, dtype=BF, scale=1.0)
    O = g.orthogonalize(G)
    for _ in range(3):
        assert torch.equal(g.orthogonalize(G), O)
    assert g.orthogonalize(G, G) is G and torch.equal(G, O)


def test_streams_and_capture(lib):
    h = lib.Gemm()
    G = update(200, 300, dtype=BF, scale=1.0)
    want = h.orthogonalize(G)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = h.orthogonalize(G)
    s.synchronize()
    by_arg = h.orthogonalize(G, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(by_arg, want)
    graph_h = lib.Gemm()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_h.orthogonalize(G, out)
    G.copy_(update(200, 300, dtype=BF, scale=2.0, seed=1))
    want = h.orthogonalize(G)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    h.close()
    graph_h.close()


def test_one_launch_on_two_streams_and_captured(lib):
    """Sizes whose products run in one launch: two handles at once, and a captured call
    beside them, give the bits of a call alone."""
    shapes = [(6, 900, 1500), (1, 4096, 4096)]
    hs = [lib.Gemm() for _ in range(3)]
    for n, shape in enumerate(shapes):
        G = update(*shape, dtype=BF, scale=1.0, kind="few")
        want = hs[0].orthogonalize(G)
        torch.cuda.synchronize()
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hs[2].orthogonalize(G, out)
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = [torch.empty_like(want) for _ in range(2)]
        for _ in range(4):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    got[i].zero_()
                    hs[i].orthogonalize(G, got[i])
            with torch.cuda.stream(streams[2]):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for h in hs:
            h.sync()
        assert torch.equal(got[0], want) and torch.equal(got[1], want) and torch.equal(out, want)
        if n == 0:
            ref = ortho.define(G[5], (3.4445, -4.7750, 2.0315))
            assert float((want[5].double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
        del graph
    for h in hs:
        h.close()


@pytest.mark.parametrize("r,c", [(64, 64), (512, 2048), (2048, 4096), (4096, 4096)])
def test_a_wait_that_runs_out(lib, r, c):
    """A load that never comes: the call gives up, says so, and the next one is right."""
    h = lib.Gemm()
    G = update(r, c, dtype=BF, scale=1.0)
    want = h.orthogonalize(G)
    h.sync()
    assert lib.gemm_debug_set(h.h, lib.GEMM_DEBUG_SKIP_FIRST_LOAD, 20_000_000) == 0
    h.orthogonalize(G)
    with pytest.raises(lib.GemmError) as e:
        h.sync()
    assert e.value.status == 5
    assert lib.gemm_debug_set(h.h, 0, 0) == 0
    assert torch.equal(h.orthogonalize(G), want)
    h.sync()
    h.close()


def test_refusals(lib, g):
    G = torch.zeros(2, 8, 16, device="cuda")
    for bad in (lambda: g.orthogonalize(G[0, 0]), lambda: g.orthogonalize(G.cpu()),
                lambda: g.orthogonalize(G, torch.zeros(2, 8, 16, device="cuda")),
                lambda: g.orthogonalize(G, torch.zeros(8, 16, device="cuda", dtype=BF)),
                lambda: g.orthogonalize(G, torch.zeros(3, 8, 16, device="cuda", dtype=BF)),
                lambda: g.orthogonalize(G.mT), lambda: g.orthogonalize(G, coefficients=(1.0, 2.0)),
                lambda: g.orthogonalize(G, steps=3, coefficients=((1.5, -0.5, 0.0),) * 2)):
        with pytest.raises(ValueError):
            bad()
    nan, inf = float("nan"), float("inf")
    for bad in (dict(steps=0), dict(steps=33), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(scale=nan),
                dict(scale=inf), dict(coefficients=(1.0, nan, 0.0)), dict(coefficients=(inf, 1.0, 0.0))):
        with pytest.raises(lib.GemmError) as e:
            g.orthogonalize(G, **bad)
        assert e.value.status == 1, bad
    with pytest.raises(lib.GemmError):
        g.orthogonalize(G[:1].expand(2, 8, 16))
    a = dict(h=g.h, batch=1, rows=8, cols=16, G=G.data_ptr(), ldg=16, stride_g=0, g_dtype=lib.GEMM_F32,
             O=G.data_ptr(), ldo=16, stride_o=0, coefficients=(1.5, -0.5, 0.0))
    for bad in (dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(batch=65536), dict(rows=65537), dict(ldg=15),
                dict(ldo=15), dict(g_dtype=3), dict(G=0), dict(O=0), dict(G=G.data_ptr() + 2), dict(O=G.data_ptr() + 1),
                dict(batch=2, stride_g=127, stride_o=128), dict(batch=2, stride_g=128, stride_o=127)):
        assert lib.ortho_update(**{**a, **bad}) == 1, bad
    assert lib.ortho_update(**{**a, "rows": 0, "G": 0, "O": 0}) == 0
