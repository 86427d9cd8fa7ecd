"""Infinities and NaN through the feed-forward operators: they reach what the
64-bit definition makes not finite, and leave everything else as it was, bit
for bit."""
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
INF, NAN = float("inf"), float("nan")
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


def same_places(got, want, what):
    """Not finite exactly where `want` is not; returns those places."""
    bad = ~torch.isfinite(want)
    assert torch.equal(~torch.isfinite(got.cpu().double()), bad), what
    return bad


def vec(gen, n, mean=1.0):
    return (torch.randn(n, generator=gen) * 0.1 + mean).cuda()


# (tensor, row, column, value) planted, one at a time
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("M,N,pair", [(700, 96, (BF, BF)), (40, 1023, (F32, BF)), (333, 4096, (BF, BF)),
                                      (20, 9001, (F32, F32)), (170, 2048, (FP, FP))])
@pytest.mark.parametrize("pre,post", [("rms", "rms"), ("layer", "layer"), ("rms", None), ("layer", "rms")])
def test_norm_rows(lib, M, N, pair, pre, post, value):
    xt, zt = pair
    gen = torch.Generator().manual_seed(M + N)
    t = {k: torch.randn(M, N, generator=gen).to(d) for k, d in (("X", xt), ("Z", zt), ("dY", zt), ("dXO", xt))}
    w = {k: vec(gen, N, m) for k, m in (("wpre", 1.0), ("bpre", 0.0), ("wpost", 1.0), ("bpost", 0.0))}
    gate = vec(gen, N, 0.5).view(1, N)

    def forward(t):
        return dict(zip(("XO", "Y"), lib.norm_block(
            t["X"].cuda(), t["Z"].cuda(), pre=pre, pre_weight=w["wpre"], pre_bias=w["bpre"], post=post,
            post_weight=w["wpost"], post_bias=w["bpost"], gate=gate, gate_rows=M, scale=0.5, eps=EPS)))

    def backward(t):
        out = {"dX": torch.empty(M, N, dtype=xt, device="cuda"), "dZ": torch.empty(M, N, dtype=zt, device="cuda"),
               "dgate": torch.empty(1, N, device="cuda")}
        out.update({k: torch.empty(N, device="cuda") for k in ("dpre_weight", "dpre_bias", "dpost_weight",
                                                               "dpost_bias")})
        lib.norm_block_backward(t["X"].cuda(), t["dY"].cuda(), t["dXO"].cuda(), t["Z"].cuda(), pre=pre,
                                pre_weight=w["wpre"], post=post, post_weight=w["wpost"], post_bias=w["bpost"],
                                gate=gate, gate_rows=M, scale=0.5, eps=EPS, **out)
        return out

    c = {k: v.cpu() for k, v in w.items()}
    cf, cb = forward(t), backward(t)
    for name in ("X", "Z"):
        p = {k: v.clone() for k, v in t.items()}
        rows = {"X": [0, M - 1], "Z": [M // 2]}[name]
        for r in rows:
            p[name][r, (r * 7) % N] = value
        got = forward(p)
        XO, _ = ref.norm_block(p["X"], p["Z"], pre, None, None, post, c["wpost"], c["bpost"], gate.cpu(), M, 0.5, EPS)
        Y, _ = ref.norm_pre(got["XO"].cpu(), pre, c["wpre"], c["bpre"], EPS)
        same_places(got["XO"], XO, "XO")
        same_places(got["Y"], Y, "Y")
        keep = [i for i in range(M) if i not in rows]
        assert torch.equal(got["XO"][keep], cf["XO"][keep]) and torch.equal(got["Y"][keep], cf["Y"][keep])
    for name in ("X", "Z", "dY", "dXO"):
        p = {k: v.clone() for k, v in t.items()}
        r, col = M - 1 if name == "Z" else M // 3, (M * 5) % N
        p[name][r, col] = value
        got = backward(p)
        want = ref.norm_block_backward(p["X"], p["dY"], p["dXO"], p["Z"], pre, c["wpre"], post, c["wpost"], c["bpost"],
                                       gate.cpu(), M, 0.5, EPS)
        for k in got:
            bad = same_places(got[k], want[k][0], (name, k))
            if k in ("dX", "dZ"):
                keep = [i for i in range(M) if i != r]
                assert torch.equal(got[k][keep], cb[k][keep]), (name, k)
            else:
                # a finite column of a row with an infinity may change (by the row's size)
                ok = ~bad
                e = want[k][1] + ref.rounding(want[k][0].abs(), got[k].dtype)
                assert ((got[k].cpu().double() - want[k][0]).abs() <= e)[ok & torch.isfinite(e)].all(), (name, k)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", None])
@pytest.mark.parametrize("M,F,K", [(40, 256, 128), (300, 129, 77), (600, 512, 256)])
def test_gated_backward_stays_in_its_row_and_column(lib, act, M, F, K):
    """What is planted at (r, c) of P or dH reaches dP there, dX's row and dW's rows."""
    g = lib.Gemm()
    gen = torch.Generator().manual_seed(M + F)
    t = {"dH": torch.randn(M, F, generator=gen).to(BF), "P": torch.randn(M, 2 * F, generator=gen).to(BF)}
    X, W = torch.randn(M, K, generator=gen).to(BF).cuda(), torch.randn(2 * F, K, generator=gen).to(BF).cuda()

    def backward(t):
        out = {"dP": torch.empty(M, 2 * F, dtype=BF, device="cuda"), "dX": torch.empty(M, K, dtype=F32, device="cuda"),
               "dW": torch.empty(2 * F, K, dtype=F32, device="cuda"), "dbias": torch.empty(2 * F, device="cuda")}
        g.glu_backward(t["dH"].cuda(), t["P"].cuda(), X, W, act=act, **out)
        g.sync()
        return {k: v.cpu() for k, v in out.items()}
    clean = backward(t)
    for name, r, c, value in (("dH", 3, 5, INF), ("dH", M - 1, F - 1, NAN), ("P", 7, 9, NAN), ("P", 7, F + 9, INF),
                              ("P", M // 2, F - 1, -INF)):
        p = {k: v.clone() for k, v in t.items()}
        p[name][r, c] = value
        got = backward(p)
        f = c % F                                        # the gate's and the up projection's column
        places = torch.zeros(M, 2 * F, dtype=torch.bool)
        places[r, f] = places[r, F + f] = True
        if act == "relu" and value == -INF:              # ReLU and its slope there are 0
            assert (got["dP"][places] == 0).all()
        else:
            assert not torch.isfinite(got["dP"][places]).all()
        assert torch.equal(got["dP"][~places], clean["dP"][~places])
        bad = ~torch.isfinite(got["dP"].double())
        for k, hit in (("dX", bad.any(1)), ("dW", bad.any(0)), ("dbias", bad.any(0))):
            touched = places.any(1) if k == "dX" else places.any(0)
            assert torch.equal(got[k][~touched], clean[k][~touched]), (name, k)
            assert (~torch.isfinite(got[k][hit])).all(), (name, k)
    g.close()


@pytest.mark.parametrize("M", [1, 2, 5, 60, 128, 300])
def test_gated_forward_stays_in_its_row(lib, M):
    """A token that is not finite spoils itself only, on every path (tails and
    padding of K included)."""
    g = lib.Gemm()
    gen = torch.Generator().manual_seed(M)
    for F, K in ((300, 128), (256, 1000), (129, 77), (1024, 520)):
        X = torch.randn(M, K, generator=gen).to(BF)
        W = torch.randn(2 * F, K, generator=gen).to(BF).cuda()
        clean = g.glu(X.cuda(), W)
        for value in (INF, NAN):
            for r, c in ((0, 0), (M - 1, K - 1)):
                p = X.clone()
                p[r, c] = value
                got = g.glu(p.cuda(), W)
                keep = [i for i in range(M) if i != r]
                assert torch.equal(got[keep], clean[keep])
                if value != value:
                    assert torch.isnan(got[r]).all()
        # a weight that is not finite spoils its column only
        V = W.clone()
        V[F + 3, K - 1] = NAN
        got = g.glu(X.cuda(), V)
        assert torch.isnan(got[:, 3]).all()
        cols = [i for i in range(F) if i != 3]
        assert torch.equal(got[:, cols], clean[:, cols])
    g.close()
