"""The orthogonalised update at the ends of its range: the longest sides and the most
matrices of a batch."""
import pytest
import torch

import ortho_model as om
import ortho_ref as ortho

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import mixed_precision_dense_sm_gb300 as lib
    h = lib.Gemm()
    yield h
    h.close()


@pytest.mark.parametrize("r,c", [(64, 65536), (65536, 64), (5, 65535), (65535, 5), (65536, 1), (1, 65536)])
def test_longest_sides(g, r, c):
    for steps in (5, 8):
        G = om.update("rank1", r, c).cuda()
        om.check(g.orthogonalize(G, steps=steps), G, steps=steps)


def test_most_matrices(g):
    gen = torch.Generator().manual_seed(3)
    G = torch.randn(65535, 3, 2, generator=gen).cuda()
    for steps in (5, 8):
        O = g.orthogonalize(G, steps=steps)
        g.sync()
        for i in (0, 1, 151, 152, 4095, 32768, 65533, 65534):
            ortho.check(O[i], G[i], steps=steps)
        assert not bool(O.isnan().any())
