"""grad_clip's argument checks where nothing would be written (no GPU)."""
import math

import pytest
import torch

import mixed_precision_dense_sm_gb300 as lib

F32, BF16 = lib.GEMM_F32, lib.GEMM_BF16


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would run on made-up addresses")
def test_the_norm_alone_takes_overlapping_tensors():
    """In place, with nothing to scale, only the norm is written: tensors may
    overlap or be listed twice.  (Status 4: accepted, but there is no device.)"""
    def clip(grads, outs=None, max_norm=math.inf, inv_scale=1.0, sizes=(4, 4), dtypes=(F32, F32)):
        return lib.grad_clip_raw(list(grads), None if outs is None else list(outs), list(sizes), list(dtypes),
                                 max_norm, inv_scale, 1 << 20, 1 << 21, 1 << 20)
    assert clip((256, 512)) == 4
    for g in ((256, 256), (256, 264)):
        assert clip(g) == 4 and clip(g, outs=g) == 4
        # whatever is scaled, or goes elsewhere, is still refused
        assert clip(g, max_norm=1.0) == 1 and clip(g, max_norm=3e38) == 1 and clip(g, inv_scale=0.5) == 1
        assert clip(g, outs=(1024, 1024)) == 1 and clip(g, outs=(g[0], 1028)) == 1
    assert clip((256, 260), sizes=(4, 4), dtypes=(F32, BF16)) == 4
    assert clip((256, 260, 8), sizes=(4, 4, 0), dtypes=(F32, BF16, F32), outs=(256, 260, 16)) == 4
