"""GPU parity of the gradient norm and clipping (grad_clip) against 64-bit
sums: one tensor to more than one launch's worth, odd sizes and alignments,
types, extreme magnitudes, in place and apart, special values, capture."""
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


def tensors(sizes, dtypes, scale=1.0, seed=0, off=0):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = torch.empty(n + off, dtype=dt)
        buf[off:] = (torch.randn(n, generator=gen) * scale).to(dt)
        out.append(buf.cuda()[off:])
    return out


def run(lib, gs, max_norm, inv_scale=1.0, in_place=False, outs=None):
    """The squares of a batch are summed in FP32: at most 8 additions in each
    of 4 sums and 2 to join them, so the norm is off by 6 roundings and its
    own; the factor adds two."""
    ins = [t.cpu().double() for t in gs]
    norm = inv_scale * math.sqrt(math.fsum(float((t * t).sum()) for t in ins))
    outs = gs if in_place else (outs or [torch.empty_like(t) for t in gs])
    got = lib.grad_clip(gs, max_norm, outputs=None if in_place else outs, inv_scale=inv_scale)
    f = inv_scale * (max_norm / norm if norm > max_norm else 1.0)
    assert abs(float(got) - norm) <= 8 * ref.U32 * norm
    for o, t in zip(outs, ins):
        r = t * f
        e = 10 * ref.U32 * r.abs()
        ref.check(o, r, e + ref.rounding(r.abs() + e, o.dtype), "out")
    return got, outs


@pytest.mark.parametrize("n", [0, 1, 7, 8, 9, 255, 4096, 16383, 16384, 16385, 100001, 3000000])
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
def test_one_tensor(lib, n, dt):
    run(lib, tensors([n], [dt]), 0.5 if n else 1.0)
    run(lib, tensors([n], [dt]), 1e30)
    run(lib, tensors([n], [dt], off=3), 0.25, in_place=True)


@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 512, 513, 1500])
def test_counts(lib, count):
    sizes = [(i * 37) % 501 for i in range(count)]
    run(lib, tensors(sizes, [BF, F32, FP]), 1.0)
    run(lib, tensors(sizes, [F32]), 1.0, inv_scale=0.125, in_place=True)


def test_mixed_alignment(lib):
    gs = tensors([1000, 70000, 33], [BF, F32, FP], off=1)
    outs = [torch.empty(t.numel() + 2, dtype=t.dtype, device="cuda")[2:] for t in gs]
    run(lib, gs, 1.0, outs=outs)


@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-20, 1e-12, 1.0, 1e15, 1e25, 1e34])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
def test_magnitudes(lib, scale, dt):
    """FP32 squares of these over- or underflow: the norm does not.  Nothing is
    clipped (a result would leave the normal range where its rounding bound holds)."""
    run(lib, tensors([5000, 100], [dt], scale=scale), 3e38)


def test_one_large_among_small(lib):
    gs = tensors([5000], [F32], scale=1e-25)
    gs[0][1234] = 3e20
    run(lib, gs, 1e30)
    gs = tensors([5000], [FP], scale=0.0)
    gs[0][77] = 2.0 ** -24                            # the smallest FP16 subnormal
    run(lib, gs, 1.0)


def test_zero_gradients(lib):
    gs = [torch.zeros(1000, dtype=BF, device="cuda")]
    got, outs = run(lib, gs, 1.0)
    assert float(got) == 0 and (outs[0] == 0).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite(lib, bad):
    gs = tensors([3000, 50], [F32])
    gs[1][13] = bad
    want = [t.clone() for t in gs]
    got = lib.grad_clip(gs, 1.0)
    assert not math.isfinite(float(got))
    assert all(torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) for a, b in zip(gs, want))


def test_norm_alone_and_determinism(lib):
    gs = tensors([1 << 20, 12345], [BF, F32])
    want = [t.clone() for t in gs]
    a = lib.grad_clip(gs, math.inf)
    assert all(torch.equal(x, y) for x, y in zip(gs, want))
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(lib.grad_clip_workspace(2), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(lib.grad_clip(gs, math.inf, norm=norm, workspace=ws), a)


def test_clipped_norm_is_max_norm(lib):
    gs = tensors([200000, 777], [F32])
    lib.grad_clip(gs, 2.0)
    # each element is off by at most 11 roundings
    assert abs(float(lib.grad_clip(gs, math.inf)) - 2.0) < 2.0 * 20 * ref.U32


def test_capture(lib):
    gs = tensors([70000, 333], [BF, F32])
    outs = [torch.empty_like(t) for t in gs]
    want, ref_outs = run(lib, gs, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = lib.grad_clip(gs, 1.0, outputs=outs)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, ref_outs))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm = lib.grad_clip(gs, 1.0, outputs=outs, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(norm, want)


def test_apart_and_in_place_in_one_list(lib):
    """Some outputs are their gradients, some lie right beside other tensors; a
    gradient listed twice counts twice."""
    flat = torch.randn(4000, device="cuda")
    gs = [flat[:1000], flat[1000:1007], flat[2000:3000], flat[1000:1007]]
    outs = [flat[:1000], torch.empty(7, device="cuda"), flat[3000:4000], torch.empty(7, device="cuda")]
    ins = [t.cpu().double() for t in gs]
    norm = math.sqrt(sum(float((t * t).sum()) for t in ins))
    got = lib.grad_clip(gs, 1.0, outputs=outs)
    assert abs(float(got) - norm) <= 8 * ref.U32 * norm
    for o, t in zip(outs, ins):
        r = t / norm
        ref.check(o, r, 11 * ref.U32 * r.abs(), "out")


def test_no_tensors(lib):
    assert float(lib.grad_clip([], 1.0)) == 0.0


def test_refusals_on_the_device(lib):
    a = torch.ones(64, device="cuda")
    for bad in (lambda: lib.grad_clip([a[::2]], 1.0), lambda: lib.grad_clip([a], 1.0, outputs=[a.to(BF)]),
                lambda: lib.grad_clip([a], 1.0, outputs=[]), lambda: lib.grad_clip([a.cpu()], 1.0)):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(max_norm=0.0), dict(max_norm=1.0, inv_scale=0.0), dict(max_norm=float("nan"))):
        with pytest.raises(lib.GemmError):
            lib.grad_clip([a], **kw)
    with pytest.raises(lib.GemmError):
        lib.grad_clip([a, a], 1.0)
    with pytest.raises(lib.GemmError):
        lib.grad_clip([a], 1.0, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
