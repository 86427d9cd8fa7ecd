"""The orthogonalised update's schedules, each against the definition and the model of
its roundings (ortho_model): X X^T by tiles of 128, 64 and 32 columns with K in one to
eight parts, wide and tall (where tiles of 128 are mirrored and others are not), on sides
that are and are not whole tiles; products on single tiles beside products on pairs."""
import pytest
import torch

import ortho_model as om

pytestmark = pytest.mark.gpu

# (batch, rows, cols): columns of a tile of the first product x parts of K, on 152 SMs
CASES = [
    # wide
    (1, 100, 500),      # 32 x 1
    (1, 400, 1500),     # 32 x 2
    (2, 257, 1411),     # 32 x 2
    (1, 256, 4096),     # 32 x 4
    (1, 129, 1205),     # 32 x 4
    (3, 400, 401),      # 64 x 1
    (1, 700, 3000),     # 64 x 2
    (1, 400, 3001),     # 64 x 4
    (4, 129, 3000),     # 64 x 4
    (1, 150, 5003),     # 64 x 8
    (16, 257, 300),     # 128 x 1
    (1, 1200, 2000),    # 128 x 2
    (2, 999, 2001),     # 128 x 2
    (1, 1000, 3001),    # 128 x 4
    (1, 1024, 8192),    # 128 x 4
    (1, 520, 3000),     # 128 x 8
    (3, 257, 3005),     # 128 x 8
    (1, 512, 16384),    # 128 x 8
    # tall
    (1, 500, 100),      # 64 x 1
    (1, 2000, 520),     # 64 x 2
    (1, 2047, 601),     # 64 x 2
    (1, 1200, 400),     # 64 x 4
    (1, 1537, 385),     # 64 x 4
    (1, 1000, 200),     # 64 x 8
    (1, 4096, 256),     # 64 x 8
    (1, 1211, 67),      # 64 x 8
    (16, 300, 257),     # 128 x 1
    (1, 2000, 1200),    # 128 x 2
    (2, 2001, 999),     # 128 x 2
    (1, 3001, 1000),    # 128 x 4
    (2, 3000, 520),     # 128 x 4
    (1, 3000, 520),     # 128 x 8
    (3, 3003, 257),     # 128 x 8
    # the last product on pairs; the first and the last
    (2, 129, 5000), (2, 5000, 129), (1, 2048, 4096), (1, 4096, 2048),
    (16, 520, 700), (16, 700, 520),
]


@pytest.fixture(scope="module")
def g():
    import mixed_precision_dense_sm_gb300 as lib
    h = lib.Gemm()
    yield h
    h.close()


@pytest.mark.parametrize("batch,r,c", CASES)
def test_schedule(g, batch, r, c):
    kinds = ("few", "rank4")
    G = torch.stack([om.update(kinds[i % 2], r, c, seed=i) for i in range(batch)]).cuda()
    O = g.orthogonalize(G)
    g.sync()
    for i in sorted({0, batch // 2, batch - 1}):
        om.check(O[i], G[i])
    if batch == 1:
        G = om.update("rank4", r, c, seed=1).cuda()
        om.check(g.orthogonalize(G), G)


@pytest.mark.parametrize("batch,r,c", [(1, 256, 4096), (1, 700, 3000), (1, 520, 3000), (1, 1000, 200), (3, 3003, 257),
                                       (2, 129, 5000), (16, 700, 520)])
def test_schedule_of_eight_steps(g, batch, r, c):
    """With X's second bytes."""
    G = torch.stack([om.update("rank4" if i == 0 else "decay4", r, c, seed=i) for i in range(batch)]).cuda()
    O = g.orthogonalize(G, steps=8)
    for i in sorted({0, batch - 1}):
        om.check(O[i], G[i], steps=8)
