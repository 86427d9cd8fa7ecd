"""GPU parity of the norms around a block (norm_block, norm_block_backward)
against their 64-bit definition: widths from one column to the widest, odd and
unaligned rows, every kind of norm and gate, types, absent parts, in place,
capture, determinism, and differences."""
import itertools

import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(BF, BF), (FP, FP), (F32, F32), (F32, FP), (F32, BF)]
EPS = 1e-5
CANARY = 77.0


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def matrix(M, N, dtype, gen, scale=1.0, mean=0.0, pad=0, off=0):
    buf = torch.full((M * (N + pad) + off,), CANARY, dtype=dtype)
    v = buf[off:].view(M, N + pad)[:, :N]
    if gen is not None:
        v.copy_((torch.randn(M, N, generator=gen) * scale + mean).to(dtype))
    dev = buf.cuda()
    return dev[off:].view(M, N + pad)[:, :N], dev


def intact(buf, M, N, pad, off):
    return bool((buf[:off] == CANARY).all()) and bool((buf[off:].view(M, N + pad)[:, N:] == CANARY).all())


def make(M, N, xt, zt, pre, post, gate_rows, seed=0, pad=0, off=0, vt=F32, bias=True):
    gen = torch.Generator().manual_seed(seed + 31 * M + N)
    c = {"M": M, "N": N, "pre": pre, "post": post, "gate_rows": gate_rows or 1, "scale": 0.5, "eps": EPS}
    c["X"], _ = matrix(M, N, xt, gen, 3.0, 0.3, pad, off)
    c["Z"], _ = matrix(M, N, zt, gen, 0.7, 0.1, pad, off)
    c["dY"], _ = matrix(M, N, zt, gen, 0.1, 0.0, pad, off)
    c["dXO"], _ = matrix(M, N, xt, gen, 0.1, 0.0, pad, off)

    def vec(scale, mean):
        return (torch.randn(N, generator=gen) * scale + mean).to(vt).cuda()
    c["wpre"], c["bpre"] = vec(0.1, 1.0), vec(0.1, 0.0) if bias else None
    c["wpost"], c["bpost"] = vec(0.1, 1.0), vec(0.1, 0.0) if bias else None
    c["gate"] = None
    if gate_rows:
        c["gate"] = (torch.randn(-(-M // gate_rows), N, generator=gen) * 0.3 + 0.5).to(vt).cuda()
    return c


def cpu(t):
    return None if t is None else t.cpu()


def run_forward(lib, c, pad=0, off=0, in_place=False):
    M, N, xt, zt = c["M"], c["N"], c["X"].dtype, c["Z"].dtype
    X0 = c["X"].cpu()
    XO, xb = (c["X"], None) if in_place else matrix(M, N, xt, None, pad=pad, off=off)
    Y, yb = matrix(M, N, zt, None, pad=pad, off=off)
    lib.norm_block(c["X"], c["Z"], XO, Y, pre=c["pre"], pre_weight=c["wpre"], pre_bias=c["bpre"],
                   post=c["post"], post_weight=c["wpost"], post_bias=c["bpost"], gate=c["gate"],
                   gate_rows=c["gate_rows"], scale=c["scale"], eps=c["eps"])
    r, t = ref.norm_block(X0, cpu(c["Z"]), c["pre"], None, None, c["post"], cpu(c["wpost"]),
                          cpu(c["bpost"]), cpu(c["gate"]), c["gate_rows"], c["scale"], c["eps"])
    ref.check(XO, r, t + ref.rounding(r.abs() + t, xt), "XO")
    r, t = ref.norm_pre(XO.cpu(), c["pre"], cpu(c["wpre"]), cpu(c["bpre"]), c["eps"])
    ref.check(Y, r, t + ref.rounding(r.abs() + t, zt), "Y")
    assert (in_place or intact(xb, M, N, pad, off)) and intact(yb, M, N, pad, off)
    return XO, Y


def run_backward(lib, c, pad=0, off=0, in_place=False, gt=F32, biases=True):
    M, N, xt, zt = c["M"], c["N"], c["X"].dtype, c["Z"].dtype
    dXO0, Z0 = cpu(c["dXO"]), cpu(c["Z"])
    dX, xb = (c["dXO"], None) if in_place else matrix(M, N, xt, None, pad=pad, off=off)
    dZ, zb = (c["Z"], None) if in_place else matrix(M, N, zt, None, pad=pad, off=off)
    v = {k: torch.full((N,), CANARY, dtype=gt, device="cuda")
         for k in ["dpre_weight", "dpost_weight"] + (["dpre_bias", "dpost_bias"] if biases else [])}
    if c["gate"] is not None:
        v["dgate"] = torch.full(c["gate"].shape, CANARY, dtype=gt, device="cuda")
    lib.norm_block_backward(c["X"], c["dY"], c["dXO"], c["Z"], pre=c["pre"], pre_weight=c["wpre"],
                            post=c["post"], post_weight=c["wpost"], post_bias=c["bpost"],
                            gate=c["gate"], gate_rows=c["gate_rows"], scale=c["scale"], eps=c["eps"],
                            dX=dX, dZ=dZ, **v)
    want = ref.norm_block_backward(cpu(c["X"]), cpu(c["dY"]), dXO0, Z0, c["pre"], cpu(c["wpre"]),
                                   c["post"], cpu(c["wpost"]), cpu(c["bpost"]), cpu(c["gate"]),
                                   c["gate_rows"], c["scale"], c["eps"])
    got = {"dX": dX, "dZ": dZ, **v}
    for k, x in got.items():
        r, t = want[k]
        ref.check(x, r, t + ref.rounding(r.abs() + t, x.dtype), k)
    assert in_place or (intact(xb, M, N, pad, off) and intact(zb, M, N, pad, off))
    return got


WIDTHS = [1, 2, 7, 8, 31, 32, 33, 100, 255, 256, 257, 264, 511, 512, 1000, 1023, 1024, 1025, 2040, 2048,
          2056, 4095, 4096, 4104, 5120, 8191, 8192, 8200, 12288, 16383, 16384]


@pytest.mark.parametrize("N", WIDTHS)
def test_widths(lib, N):
    for (xt, zt), kind in zip(PAIRS, itertools.cycle(["rms", "layer"])):
        c = make(37, N, xt, zt, kind, kind, 10)
        run_forward(lib, c)
        run_backward(lib, c)


@pytest.mark.parametrize("M", [1, 2, 3, 63, 300, 305, 700, 4999])
def test_row_counts(lib, M):
    for N, rows in ((96, 1), (1024, 100), (4096, M)):
        c = make(M, N, BF, BF, "rms", "layer", rows)
        run_forward(lib, c)
        run_backward(lib, c)


@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("rows", [0, 1, 2, 19, 50, 1000])
def test_kinds_and_gates(lib, pre, post, rows):
    c = make(50, 520, F32, BF, pre, post, rows, vt=BF)
    run_forward(lib, c)
    run_backward(lib, c, gt=BF)
    run_backward(lib, c, biases=False)
    c["bpost"] = c["wpost"] = c["wpre"] = c["bpre"] = None
    run_forward(lib, c)
    run_backward(lib, c, biases=False)


# every width of a row group, for few rows and for many; the kinds that have
# kernels of their own, and RMSNorm with biases and LayerNorm without, which do not
@pytest.mark.parametrize("N", [40, 99, 256, 500, 512, 1016, 1023, 2048, 3000, 4096, 4097, 5120, 8192, 9001, 12288])
@pytest.mark.parametrize("M", [20, 340])
def test_kinds_by_width(lib, M, N):
    kinds = [("rms", "rms", False), ("rms", None, False), ("layer", "layer", True), ("layer", None, True),
             ("rms", "rms", True), ("layer", "layer", False)]
    for i, (pre, post, bias) in enumerate(kinds):
        xt, zt = PAIRS[(i + N + M) % len(PAIRS)]
        c = make(M, N, xt, zt, pre, post, (0, M, 100)[(i + N) % 3], bias=bias)
        if post is None:
            c["bpost"] = None
        run_forward(lib, c)
        run_backward(lib, c, biases=bias)


def test_many_gate_groups(lib):
    for M, rows in ((2000, 3), (2000, 100), (2000, 150), (5000, 2), (4000, 4), (4100, 4)):
        run_backward(lib, make(M, 264, BF, BF, "rms", "layer", rows))
        run_backward(lib, make(M, 33, F32, BF, "layer", "rms", rows, bias=False), biases=False)


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (0, 1), (16, 3)])
@pytest.mark.parametrize("pair", PAIRS, ids=str)
def test_strides(lib, pad, off, pair):
    for N in (264, 1023, 4096):
        c = make(29, N, *pair, "layer", "rms", 10, pad=pad, off=off, vt=FP)
        run_forward(lib, c, pad, off)
        run_backward(lib, c, pad, off, gt=FP)


@pytest.mark.parametrize("N", [96, 1023, 4096, 9000])
def test_in_place(lib, N):
    c = make(333, N, F32, BF, "rms", "layer", 100)
    run_forward(lib, c, in_place=True)
    run_backward(lib, c, in_place=True)


def test_unaligned_vectors(lib):
    c = make(40, 520, BF, BF, "layer", "layer", 7)
    for k in ("wpre", "bpre", "wpost", "bpost"):
        buf = torch.empty(521, device="cuda")
        buf[1:].copy_(c[k])
        c[k] = buf[1:]
    buf = torch.empty(c["gate"].shape[0], 523, device="cuda")
    buf[:, 2:522].copy_(c["gate"])
    c["gate"] = buf[:, 2:522]
    run_forward(lib, c)
    run_backward(lib, c)


def test_absent_parts(lib):
    c = make(70, 640, F32, BF, "rms", "rms", 0)
    none, Y = lib.norm_block(c["X"], pre="layer", pre_weight=c["wpre"], pre_bias=c["bpre"], eps=EPS)
    r, t = ref.norm_pre(c["X"].cpu(), "layer", c["wpre"].cpu(), c["bpre"].cpu(), EPS)
    assert none is None and Y.dtype == F32
    ref.check(Y, r, t + ref.rounding(r.abs() + t, F32), "Y alone")
    XO, none = lib.norm_block(c["X"], c["Z"], pre=None, post="rms", eps=EPS)
    assert none is None
    r, t = ref.norm_block(c["X"].cpu(), c["Z"].cpu(), None, None, None, "rms", None, None, None, 1, 1.0, EPS)
    ref.check(XO, r, t + ref.rounding(r.abs() + t, F32), "XO alone")
    # gradients one at a time are the same bits as all together
    whole = run_backward(lib, c)
    for k in ("dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias", "dX", "dZ"):
        out = torch.empty_like(whole[k])
        lib.norm_block_backward(c["X"], c["dY"], c["dXO"], c["Z"], pre="rms", pre_weight=c["wpre"],
                                post="rms", post_weight=c["wpost"], post_bias=c["bpost"],
                                scale=c["scale"], eps=EPS, **{k: out})
        assert torch.equal(out, whole[k]), k
    # dY or dXO absent read as zero, and a norm without a block
    for dY, dXO in ((None, c["dXO"]), (c["dY"], None)):
        dX, dZ = torch.empty_like(c["X"]), torch.empty_like(c["Z"])
        lib.norm_block_backward(c["X"], dY, dXO, c["Z"], pre="rms", post="layer", eps=EPS, dX=dX, dZ=dZ)
        w = ref.norm_block_backward(c["X"].cpu(), cpu(dY), cpu(dXO), c["Z"].cpu(), "rms", None, "layer",
                                    None, None, None, 1, 1.0, EPS)
        for x, k in ((dX, "dX"), (dZ, "dZ")):
            r, t = w[k]
            ref.check(x, r, t + ref.rounding(r.abs() + t, x.dtype), k)
    dX, dw = torch.empty_like(c["X"]), torch.empty(640, device="cuda")
    lib.norm_block_backward(c["X"], c["dY"], None, pre="layer", pre_weight=c["wpre"], eps=EPS, dX=dX,
                            dpre_weight=dw)
    w = ref.norm_block_backward(c["X"].cpu(), c["dY"].cpu(), None, None, "layer", c["wpre"].cpu(), None,
                                None, None, None, 1, 1.0, EPS)
    for x, k in ((dX, "dX"), (dw, "dpre_weight")):
        r, t = w[k]
        ref.check(x, r, t + ref.rounding(r.abs() + t, x.dtype), k)


def test_empty(lib):
    X = torch.empty(0, 64, dtype=BF, device="cuda")
    XO, Y = lib.norm_block(X, X.clone(), post="rms")
    assert XO.shape == Y.shape == (0, 64)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    lib.norm_block_backward(X, X.clone(), X.clone(), X.clone(), post="rms", dpre_weight=dw, dpost_bias=db)
    assert (dw == 0).all() and (db == 0).all()
    E = torch.empty(5, 0, dtype=BF, device="cuda")
    assert lib.norm_block(E, E.clone())[1].shape == (5, 0)


def test_special_rows(lib):
    """A row of zeros stays finite (eps), a row with a NaN or an infinity
    spoils itself only."""
    X = torch.randn(6, 512).to(BF)
    X[1] = 0
    X[2, 17] = float("nan")
    X[4, 5] = float("inf")
    for kind in ("rms", "layer"):
        _, Y = lib.norm_block(X.cuda(), pre=kind)
        Y = Y.float().cpu()
        assert (Y[1] == 0).all() and torch.isnan(Y[2]).all()
        assert torch.isnan(Y[4, 5]) and torch.isfinite(Y[[0, 1, 3, 5]]).all()


def test_constant_shift_keeps_the_variance(lib):
    """LayerNorm of values far from zero: the variance comes from deviations."""
    X = (torch.randn(8, 4096) + 4096.0)
    _, Y = lib.norm_block(X.cuda(), pre="layer", eps=1e-5)
    r, t = ref.norm_pre(X, "layer", None, None, 1e-5)
    ref.check(Y, r, t, "Y")
    # the mean's FP32 error (about 2^-12 * a few roundings) is all that is left
    assert (Y.cpu().double() - r).abs().max() < 2.0 ** -8


def test_repeats_bit_for_bit(lib):
    c = make(5000, 1024, BF, BF, "rms", "rms", 5000)
    a = run_backward(lib, c)
    b = run_backward(lib, c)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_differences(lib):
    """Gradients of sum(Y R + XO S) by central differences of the 64-bit
    definition (FP32 stream, so XO's rounding is below the step's error)."""
    gen = torch.Generator().manual_seed(9)
    M, N, h = 4, 24, 1e-5
    x, z, R, S = (torch.randn(M, N, generator=gen) for _ in range(4))
    wp, bp, wq = torch.rand(N, generator=gen) + 0.5, torch.randn(N, generator=gen), torch.rand(N, generator=gen)
    gate = torch.rand(2, N, generator=gen)
    for pre, post in (("rms", "layer"), ("layer", "rms")):
        def loss(x, z, wq, wp, bp, gate):
            xo, _ = ref.norm_block(x, z, None, None, None, post, wp, bp, gate, 2, 0.5, EPS)
            return float((ref.norm_pre(xo, pre, wq, None, EPS)[0] * R.double()).sum() + (xo * S.double()).sum())
        args = [t.double() for t in (x, z, wq, wp, bp, gate)]
        num = []
        for i, a in enumerate(args):
            n = torch.zeros_like(a)
            for j in range(a.numel()):
                hi, lo = [t.clone() for t in args], [t.clone() for t in args]
                hi[i].view(-1)[j] += h
                lo[i].view(-1)[j] -= h
                n.view(-1)[j] = (loss(*hi) - loss(*lo)) / (2 * h)
            num.append(n)
        d = [t.cuda() for t in (x, z, wq, wp, bp, gate)]
        XO, _ = lib.norm_block(d[0], d[1], pre=pre, pre_weight=d[2], post=post, post_weight=d[3],
                               post_bias=d[4], gate=d[5], gate_rows=2, scale=0.5, eps=EPS)
        out = [torch.empty_like(t) for t in d]
        lib.norm_block_backward(XO, R.cuda(), S.cuda(), d[1], pre=pre, pre_weight=d[2], post=post,
                                post_weight=d[3], post_bias=d[4], gate=d[5], gate_rows=2, scale=0.5,
                                eps=EPS, dX=out[0], dZ=out[1], dpre_weight=out[2], dpost_weight=out[3],
                                dpost_bias=out[4], dgate=out[5])
        for a, b in zip(out, num):
            # FP32 arithmetic, and differences good to about 1e-6
            assert (a.cpu().double() - b).abs().max() < 2e-5 * max(1.0, float(b.abs().max()))


def test_capture_and_streams(lib):
    c = make(200, 1024, BF, BF, "rms", "rms", 50)
    outs = {k: torch.empty_like(c[v]) for k, v in (("dX", "X"), ("dZ", "Z"), ("dgate", "gate"),
                                                   ("dpre_weight", "wpre"))}
    XO, Y = torch.empty_like(c["X"]), torch.empty_like(c["Z"])

    def step(stream=None):
        lib.norm_block(c["X"], c["Z"], XO, Y, post="rms", gate=c["gate"], gate_rows=50, pre_weight=c["wpre"],
                       stream=stream)
        lib.norm_block_backward(XO, c["dY"], c["dXO"], c["Z"], post="rms", gate=c["gate"], gate_rows=50,
                                pre_weight=c["wpre"], stream=stream, **outs)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (XO, Y, *outs.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (XO, Y, *outs.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (XO, Y, *outs.values())))
    s = torch.cuda.Stream()
    for t in (XO, Y, *outs.values()):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (XO, Y, *outs.values())))


def test_refusals_on_the_device(lib):
    X = torch.randn(4, 64, device="cuda").to(BF)
    w = torch.ones(64, device="cuda")
    for bad in (lambda: lib.norm_block(X, XO=X), lambda: lib.norm_block(X, X[:, :32]),
                lambda: lib.norm_block(X, pre_weight=w[:32]), lambda: lib.norm_block(X.cpu()),
                lambda: lib.norm_block(X, X, gate=torch.ones(3, 64, device="cuda"), gate_rows=4),
                lambda: lib.norm_block(X, pre_weight=w, pre_bias=w.to(BF)),
                lambda: lib.norm_block_backward(X, X, dgate=w.view(1, 64))):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(2, lib.NORM_MAX_N + 8, dtype=BF, device="cuda")
    with pytest.raises(lib.GemmError) as e:
        lib.norm_block(wide)
    assert e.value.status == 2
    with pytest.raises(lib.GemmError):
        lib.norm_block_backward(X, X, dpre_weight=w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
