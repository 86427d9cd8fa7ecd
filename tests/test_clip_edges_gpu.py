"""grad_clip at the ends of what it accepts."""
import math

import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def test_the_norm_alone_over_overlapping_views(lib):
    """Nothing is written: a tensor counts as often as it is listed.  (8 FP32
    roundings, as for tensors apart.)"""
    flat = torch.randn(100000, generator=torch.Generator().manual_seed(2)).cuda()
    keep = flat.clone()
    for views in ([flat, flat], [flat[:60000], flat[40000:]], [flat[i:i + 300] for i in range(0, 99000, 100)]):
        want = math.sqrt(sum(float(v.cpu().double().square().sum()) for v in views))
        for outs in (None, views):
            got = float(lib.grad_clip(views, math.inf, outputs=outs))
            assert abs(got - want) <= 8 * ref.U32 * want
        with pytest.raises(lib.GemmError) as e:
            lib.grad_clip(views, 1.0)
        assert e.value.status == 1
    assert torch.equal(flat, keep)
