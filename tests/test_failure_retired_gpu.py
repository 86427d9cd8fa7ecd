"""A wait that runs out in a captured graph whose workspace the handle has
outgrown since: the counters there are cleared too, so that other graphs on the
same buffer stay right.  (The planted missing load of gemm_debug_set; every wait
is bounded.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("M,N,K", [(64, 4096, 8192), (6272, 512, 4608)], ids=["skinny", "pairs"])
def test_timeout_in_an_outgrown_workspace(M, N, K):
    import mixed_precision_dense_sm_gb300 as lib
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    st, plan = lib.gemm_plan_query("N", "T", M, N, K, 1.0, 256, K, 256, K, 0.0, 256, N,
                                   (lib.GEMM_BF16, lib.GEMM_BF16, lib.GEMM_F32), num_sms=sms)
    assert st == 0 and plan["sk_len"] > 0 and plan["workspace_bytes"] > 0, plan
    gen = torch.Generator().manual_seed(M)
    A, B = torch.randn(M, K, generator=gen).to(BF).cuda(), torch.randn(N, K, generator=gen).to(BF).cuda()
    C, D = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    h = lib.Gemm()
    h(A, B, C, transB="T")
    h.sync()
    want = C.clone()
    good, late = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(good):
        h(A, B, C, transB="T")
    assert lib.gemm_debug_set(h.h, lib.GEMM_DEBUG_SKIP_FIRST_LOAD, 20_000_000) == 0
    with torch.cuda.graph(late):
        h(A, B, D, transB="T")
    assert lib.gemm_debug_set(h.h, 0, 0) == 0
    # unaligned rows are copied to the workspace: larger than the graphs' one
    odd = torch.randn(4 * M + 4096, K + 1, device="cuda").to(BF)
    h(odd, odd, torch.empty(odd.shape[0], odd.shape[0], device="cuda"), transB="T")
    h.sync()
    for _ in range(2):
        late.replay()
        with pytest.raises(lib.GemmError) as e:
            h.sync()
        assert e.value.status == 5
        for _ in range(3):
            C.zero_()
            good.replay()
            h.sync()
            assert torch.equal(C, want)
    del good, late
    h.close()
