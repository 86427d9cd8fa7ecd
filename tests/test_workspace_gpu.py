"""The first calls of a handle on a stream that does not wait for the default
one, which is busy meanwhile."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_first_calls_beside_a_busy_default_stream():
    import mixed_precision_dense_sm_gb300 as lib
    gen = torch.Generator().manual_seed(1)
    M, N, K = 64, 4096, 8192                              # stream-K: tile counters
    A, B = torch.randn(M, K, generator=gen).to(BF).cuda(), torch.randn(N, K, generator=gen).to(BF).cuda()
    X, W = torch.randn(300, 1001, generator=gen).to(BF).cuda(), torch.randn(512, 1001, generator=gen).to(BF).cuda()
    first = lib.Gemm()
    want, wantH = torch.empty(M, N, device="cuda"), first.glu(X, W)
    first(A, B, want, transB="T")
    first.sync()
    busy = torch.randn(4096, 4096, device="cuda").to(BF)
    side = torch.cuda.Stream()
    for _ in range(5):
        h = lib.Gemm()
        C, H = torch.zeros_like(want), torch.zeros_like(wantH)
        torch.cuda.synchronize()
        for _ in range(100):
            busy @ busy
        h(A, B, C, transB="T", stream=side.cuda_stream)
        h.glu(X, W, H, stream=side.cuda_stream)
        h(A, B, C, transB="T", stream=side.cuda_stream)
        h.sync(side.cuda_stream)
        assert torch.equal(C, want) and torch.equal(H, wantH)
        torch.cuda.synchronize()
        h.close()
    first.close()
