"""The gated layer at the longest rows that are not 16-byte aligned: zeros but
for the first and the last elements, whose products are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def need(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def test_unaligned_k():
    import mixed_precision_dense_sm_gb300 as lib
    need(80)
    M, K, F = 3, 2 ** 31 - 1, 1
    g = lib.Gemm()
    X, W = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(2 * F, K, dtype=BF, device="cuda")
    for t in (X, W):
        t[:, :8] = 2
        t[:, -8:] = torch.arange(1, 9, device="cuda").to(BF)
    W[1] *= -1
    H = g.glu(X, W, act="none")
    g.sync()
    P = 8 * 4 + sum(i * i for i in range(1, 9))            # 236
    assert (H.float() == torch.tensor(-P * P, dtype=torch.float32).to(BF).float()).all()
    g.close()
    del X, W
    torch.cuda.empty_cache()


def test_backward_of_the_widest_layer():
    """2F = 2^31 - 2 unaligned columns of P: dX's product runs over all of them."""
    import mixed_precision_dense_sm_gb300 as lib
    need(120)
    M, K, F = 1, 8, 2 ** 30 - 1
    g = lib.Gemm()
    dH, P = torch.zeros(M, F, dtype=BF, device="cuda"), torch.zeros(M, 2 * F, dtype=BF, device="cuda")
    W = torch.zeros(2 * F, K, dtype=BF, device="cuda")
    dH[:, -3:], P[:, F - 3:F], P[:, -3:] = 1, 2, 3         # dG = dH U = 3, dU = dH G = 2
    dH[:, 0], P[:, 0], P[:, F] = 1, 4, 5
    W[F - 3:F], W[-3:], W[0], W[F] = 1, 2, 3, 4
    dX = torch.empty(M, K, dtype=torch.float32, device="cuda")
    dP = g.glu_backward(dH, P, None, W, act="none", dX=dX)
    g.sync()
    assert (dX == 3 * 3 * 1 + 3 * 2 * 2 + 5 * 3 + 4 * 4).all()
    assert (dP[:, -3:] == 2).all() and (dP[:, F - 3:F] == 3).all() and int(torch.count_nonzero(dP)) == 8
    g.close()
    del dH, P, W, dP
    torch.cuda.empty_cache()
