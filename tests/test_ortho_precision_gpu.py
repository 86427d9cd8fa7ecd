"""The precision of the orthogonalised update before its result is rounded to BF16, on
spectra from rank 1 to noise and for more steps than five (ortho_model): both
orientations, single tiles and CTA pairs, X's second bytes in results of every alignment,
pitch and width, in place, batches, captured."""
import pytest
import torch

import ortho_model as om
import ortho_ref as ortho

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


@pytest.fixture(scope="module")
def g(lib):
    h = lib.Gemm()
    yield h
    h.close()


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("kind", om.KINDS)
@pytest.mark.parametrize("r,c", [(256, 1024), (1024, 256), (200, 333), (700, 129)])
def test_spectra(g, r, c, kind, steps):
    G = om.update(kind, r, c).cuda()
    om.check(g.orthogonalize(G, steps=steps), G, steps=steps, most=om.PROMISE[steps])


@pytest.mark.parametrize("steps", [1, 2, 3, 6, 7, 10])
def test_numbers_of_steps(g, steps):
    for kind in ("rank4", "decay4", "noise"):
        G = om.update(kind, 300, 520).cuda()
        om.check(g.orthogonalize(G, steps=steps), G, steps=steps)


def test_other_coefficients(g):
    for abc, steps in (((1.5, -0.5, 0.0), 20), ((2.0, -1.5, 0.5), 12),
                       ((om.MUON,) * 6 + ((2.0, -1.5, 0.5),) * 2, 8)):
        for kind in ("rank4", "few"):
            G = om.update(kind, 300, 520).cuda()
            om.check(g.orthogonalize(G, steps=steps, coefficients=abc, scale=0.2), G, abc, scale=0.2, steps=steps)


def test_stored_in_bf16(g):
    for kind in ("rank1", "rank4"):
        G = om.update(kind, 256, 1024, dtype=BF).cuda()
        for steps in (5, 8):
            om.check(g.orthogonalize(G, steps=steps), G, steps=steps, most=om.PROMISE[steps])


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("r,c", [(1500, 3000), (3000, 1500), (2048, 2047)])
def test_on_pairs(g, r, c, steps):
    """One launch for all products, without and with second bytes."""
    G = torch.stack([om.update(k, r, c) for k in ("rank4", "few")]).cuda()
    O = g.orthogonalize(G, steps=steps)
    for i in range(2):
        om.check(O[i], G[i], steps=steps, most=om.PROMISE[5] if steps == 5 else None)


@pytest.mark.parametrize("n", [1, 2, 6, 7, 8, 9, 15, 16, 17, 23, 24, 31, 33, 40])
def test_narrow(g, n):
    """Columns few enough that X's second bytes fill the result's rows, and their transposes."""
    for r, c in ((-(-40000 // n), n), (n, -(-40000 // n))):
        G = om.update("rank1", r, c).cuda()
        om.check(g.orthogonalize(G, steps=8), G, steps=8)


@pytest.mark.parametrize("c", [4, 15, 16, 17, 130, 264])
@pytest.mark.parametrize("pad,off", [(0, 0), (1, 0), (0, 1), (0, 2), (0, 3), (5, 7), (8, 8)])
def test_second_bytes_stay_in_the_result(g, c, pad, off):
    """Padding between the rows and what lies around the result keep their values; the
    result does not depend on where it lies."""
    r, batch = 150, 3
    G = torch.stack([om.update("rank1", r, c, seed=i) for i in range(batch)]).cuda()
    want = g.orthogonalize(G, steps=8)
    buf = torch.full((off + (batch * r + 2) * (c + pad) + 9,), 9.0, dtype=BF, device="cuda")
    out = buf[off:off + batch * (r * (c + pad))].view(batch, r, c + pad)[:, :, :c]
    hull = buf.clone()
    g.orthogonalize(G, out, steps=8)
    assert torch.equal(out, want)
    out.fill_(9.0)
    assert torch.equal(buf, hull), "padding"


def test_in_place_and_apart(g):
    """The result over the update it comes from, and over the update of another matrix."""
    for r, c in ((200, 300), (300, 12)):
        G = om.update("rank4", r, c, dtype=BF).cuda()
        want = g.orthogonalize(G, steps=8)
        both = torch.stack([G, G])
        shifted = both.flatten()[5:5 + r * c].view(r, c)
        shifted.copy_(G)
        # (the result begins five elements before the update)
        assert torch.equal(g.orthogonalize(shifted, both[0], steps=8), want)
        assert g.orthogonalize(G, G, steps=8) is G and torch.equal(G, want)


def test_batches_and_special_values(g):
    G = torch.stack([om.update(k, 150, 270) for k in ("rank1", "rank4", "decay6", "noise", "few")]).cuda()
    O = g.orthogonalize(G, steps=8)
    for i in range(5):
        om.check(O[i], G[i], steps=8)
    Z = G.clone()
    Z[0], Z[2, 3, 4], Z[4, 0, 0] = 0.0, float("inf"), float("nan")
    got = g.orthogonalize(Z, steps=8)
    assert not got[0].any() and bool(got[2].isnan().all()) and bool(got[4].isnan().all())
    assert torch.equal(got[1], O[1]) and torch.equal(got[3], O[3])


def test_same_bits_and_capture(lib):
    for shape in ((300, 700), (2, 1500, 1600)):
        h, graph_h = lib.Gemm(), lib.Gemm()
        G = om.update("rank4", shape[-2], shape[-1]).expand(*shape).contiguous().cuda()
        want = h.orthogonalize(G, steps=8)
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graph_h.orthogonalize(G, out, steps=8)
        s = torch.cuda.Stream()
        for _ in range(3):
            graph.replay()
            with torch.cuda.stream(s):
                assert torch.equal(h.orthogonalize(G, steps=8), want)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            out.fill_(float("nan"))
        for x in (h, graph_h):
            x.sync()
        del graph
        h.close()
        graph_h.close()


@pytest.mark.parametrize("r,c", [(200, 400), (4096, 4096)])
def test_a_wait_that_runs_out(lib, r, c):
    """With second bytes as well: the call gives up, says so, and the next one is right."""
    h = lib.Gemm()
    G = om.update("rank4", r, c, dtype=BF).cuda()
    want = h.orthogonalize(G, steps=8)
    h.sync()
    assert lib.gemm_debug_set(h.h, lib.GEMM_DEBUG_SKIP_FIRST_LOAD, 20_000_000) == 0
    h.orthogonalize(G, steps=8)
    with pytest.raises(lib.GemmError) as e:
        h.sync()
    assert e.value.status == 5
    assert lib.gemm_debug_set(h.h, 0, 0) == 0
    assert torch.equal(h.orthogonalize(G, steps=8), want)
    h.sync()
    h.close()
