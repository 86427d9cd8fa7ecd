"""grad_clip at the ends of what it accepts."""
import math

import pytest
import torch

import ffn_ref as ref
import test_grad_gpu as clip

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


@pytest.mark.parametrize("inv_scale", [1.0, 0.5])
def test_a_norm_above_fp32(lib, inv_scale):
    """Finite gradients whose norm FP32 does not hold: the caller sees an infinite
    norm, and nothing is clipped (inv_scale applies, exactly where a power of two)."""
    for n, v in ((2, 3e38), (1000, -1.0e38), (40, 3.38e38)):
        g = torch.full((n,), v, device="cuda")
        want = g * inv_scale
        if inv_scale * math.sqrt(n) * abs(v) <= torch.finfo(F32).max:
            continue
        for in_place in (False, True):
            t, out = g.clone(), torch.zeros_like(g)
            got = lib.grad_clip([t], 1.0, outputs=None if in_place else [out], inv_scale=inv_scale)
            assert math.isinf(float(got))
            assert torch.equal(t if in_place else out, want)
    g = torch.full((4,), 1.7e38, device="cuda")                   # 3.4e38: the largest that FP32 holds
    got = lib.grad_clip([g], 1.0)
    assert abs(float(got) - 3.4e38) <= 8 * ref.U32 * 3.4e38 and torch.allclose(g, torch.full_like(g, 0.5))


# the factor max_norm / norm: normal, subnormal in FP32, below all of FP32
@pytest.mark.parametrize("max_norm", [1e-5, 1e-6, 1e-8, 1e-10, 1e-12, 1e-13, 1e-16])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
def test_factors_below_the_normal_range(lib, dt, max_norm):
    """Elements of about 1e30 clipped to a small norm stay normal numbers, though
    the factor is not one: the same bound as for any other factor."""
    gs = clip.tensors([5000, 100, 7], [dt], scale=1e30, off=1)
    clip.run(lib, gs, max_norm)
    clip.run(lib, gs, max_norm, inv_scale=0.5, outs=[torch.empty(t.numel() + 2, dtype=dt, device="cuda")[2:]
                                                     for t in gs])
    clip.run(lib, gs, max_norm, in_place=True)


def test_a_small_scale_and_clipping(lib):
    """inv_scale = 2^-140, a subnormal: exact where nothing is clipped, a bound as ever where it is."""
    clip.run(lib, clip.tensors([3000], [F32], scale=1e34), 1e30, inv_scale=2.0 ** -140)
    clip.run(lib, clip.tensors([3000], [F32], scale=1e34), 1e-7, inv_scale=2.0 ** -140)
