"""Plain 64-bit definitions of the feed-forward operators (gated linear layer,
norms around a block, gradient clipping) on CPU tensors, and the bounds their
tests use.

Error model.  A rounding to type t is off by at most half a step,
eps(t) / 2 relative, plus half of t's smallest subnormal.  FP32 arithmetic of
n dependent roundings is off by at most n 2^-24 (first order) of the sum of
the magnitudes it adds."""
import math

import torch

U32 = 2.0 ** -24


def rounding(ref, dtype):
    """Most a rounding of `ref` (64-bit tensor) to dtype can be off."""
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def check(got, ref, tol, what):
    """|got - ref| <= tol elementwise; NaN and infinities where ref has them."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(got)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = ((got - ref).abs() <= tol) | nan | inf
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off; first at {i}: got "
                             f"{got.flatten()[i].item()!r}, want {ref.flatten()[i].item()!r}, tol "
                             f"{(tol.flatten()[i] if torch.is_tensor(tol) else tol)!r}")


# ------------------------------------------------------------ gated linear layer

def act64(name, x):
    """(act, act', bound on the kernels' relative error of act, absolute error of act')."""
    if name == "silu":
        s = torch.sigmoid(x)
        rel = x.abs() * 2.0 ** -23 + 2.0 ** -20
        return x * s, s * (1 + x * (1 - s)), rel, rel * (1 + 2 * x.abs())
    if name == "gelu":
        phi = torch.special.ndtr(x)
        pdf = torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        rel = (x * x / 2 + 2) * 2.0 ** -21 + 3e-7
        return x * phi, phi + x * pdf, rel, 2 * rel
    if name == "relu":
        return torch.where(x > 0, x, x * 0), (x > 0).double(), torch.zeros_like(x), torch.zeros_like(x)
    return x, torch.ones_like(x), torch.zeros_like(x), torch.zeros_like(x)


def glu_forward(X, W, act, bias, h_dtype):
    """(H, tolerance, P, tolerance) in 64 bits.  A product's FP32 accumulation is
    off by at most 1e-5 sum|x w| + 1e-6 (the GEMM's own bound); H's error is
    that of act(g) u for g and u within it (|act'| <= 1.13), the activation's
    own, and the rounding."""
    F = W.shape[0] // 2
    X, W = X.double(), W.double()
    P = X @ W.t()
    eP = 1e-5 * (X.abs() @ W.abs().t()) + 1e-6
    if bias is not None:
        P = P + bias.double()
        eP = eP + 2 * U32 * (P.abs() + bias.double().abs())
    G, U, eg, eu = P[:, :F], P[:, F:], eP[:, :F], eP[:, F:]
    a, _, rel, _ = act64(act, G)
    H = a * U
    ea = 1.13 * eg + rel * (a.abs() + 1.13 * eg)
    eH = ea * (U.abs() + eu) + a.abs() * eu + 2 * U32 * H.abs()
    return H, eH + rounding(H.abs() + eH, h_dtype), P, eP + rounding(P.abs() + eP, h_dtype)


def glu_backward(dH, P, X, W, act, dtype, dx_dtype, dw_dtype, beta_w=0.0, dW0=None):
    """{name: (value, tolerance)}: dP, dX, dW, dbias.  The products see dP
    rounded, so they carry its error through |W| and |X|."""
    F = dH.shape[1]
    dH, P = dH.double(), P.double()
    a, d, rel, ed = act64(act, P[:, :F])
    U = P[:, F:]
    dP = torch.cat([dH * U * d, dH * a], 1)
    e32 = torch.cat([(dH * U).abs() * (ed + 4 * U32 * d.abs()), dH.abs() * a.abs() * (rel + 2 * U32)], 1)
    e = e32 + rounding(dP.abs() + e32, dtype)
    out = {"dP": (dP, e)}
    # column sums: FP32 additions of M values
    n = dP.shape[0] + 8
    out["dbias"] = (dP.sum(0), e32.sum(0) + n * U32 * dP.abs().sum(0) + 1e-30)
    if W is not None:
        Wd = W.double()
        r = dP @ Wd
        t = e @ Wd.abs() + 1e-5 * ((dP.abs() + e) @ Wd.abs()) + 1e-6
        out["dX"] = (r, t + rounding(r.abs() + t, dx_dtype))
    if X is not None:
        Xd = X.double()
        r = dP.t() @ Xd
        t = e.t() @ Xd.abs() + 1e-5 * ((dP.abs() + e).t() @ Xd.abs()) + 1e-6
        if beta_w:
            r = r + beta_w * dW0.double()
            t = t + 1e-5 * (beta_w * dW0.double()).abs()
        out["dW"] = (r, t + rounding(r.abs() + t, dw_dtype))
    return out


# ------------------------------------------------------------- norms around a block

# FP32 roundings on the way to an element: sums over a row take at most 16
# additions in a thread, 5 in its warp, 5 over the warps and 1 over a CTA
# pair; a result depends on at most three such sums (mean, size, the
# Jacobian's) and some ten products.
C32 = 128 * U32


def norm64(kind, v, eps):
    """(xhat, r, magnitude that FP32 errors of xhat are relative to)."""
    if kind in (None, "none"):
        return v, torch.ones_like(v[:, :1]), v.abs()
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - m
    r = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    mag = (v.abs() + (v.abs().mean(1, keepdim=True) if kind == "layer" else 0)) * r
    # an error of the mean also enters the size through sum d * error: second
    # order for the exact mean, bounded by mag times itself
    return d * r, r, mag * (1 + (mag.mean(1, keepdim=True) if kind == "layer" else 0))


def norm_block(X, Z, pre, wpre, bpre, post, wpost, bpost, gate, gate_rows, scale, eps):
    """XO and its tolerance before rounding, in 64 bits."""
    M, N = X.shape
    zhat, _, mag = norm64(post, Z.double(), eps)
    w = 1.0 if wpost is None else wpost.double()
    b = torch.zeros(N, dtype=torch.float64) if bpost is None else bpost.double()
    g = scale * (torch.ones(M, N, dtype=torch.float64) if gate is None
                 else gate.double().repeat_interleave(gate_rows, 0)[:M])
    n = zhat * w + b
    en = C32 * (mag * (w if isinstance(w, float) else w.abs()) + b.abs())
    XO = X.double() + g * n
    return XO, g.abs() * en + C32 * (X.double().abs() + (g * n).abs())


def norm_pre(XO, pre, wpre, bpre, eps):
    """Y of a stored XO, and its tolerance before rounding."""
    xhat, _, mag = norm64(pre, XO.double(), eps)
    w = torch.ones(XO.shape[1], dtype=torch.float64) if wpre is None else wpre.double()
    b = torch.zeros(XO.shape[1], dtype=torch.float64) if bpre is None else bpre.double()
    return xhat * w + b, C32 * (mag * w.abs() + b.abs())


def jacobian(kind, hat, r, mag, g, eg):
    """(J^T g, bound): r (g - mean(g) - hat mean(g hat)), without the parts the kind lacks."""
    if kind in (None, "none"):
        return g, eg
    N = hat.shape[1]
    dot = (g * hat).mean(1, keepdim=True)
    mdot = ((g.abs() + eg) * mag).mean(1, keepdim=True)
    v = g - hat * dot
    t = C32 * (g.abs() + mag * mdot) + eg + mag * (eg * mag).mean(1, keepdim=True)
    if kind == "layer":
        v = v - g.mean(1, keepdim=True)
        t = t + C32 * g.abs().mean(1, keepdim=True) + eg.mean(1, keepdim=True)
    return r * v, r * t + C32 * r * mag * mdot


def norm_block_backward(XO, dY, dXO, Z, pre, wpre, post, wpost, bpost, gate, gate_rows, scale, eps):
    """{name: (value, tolerance before rounding)}."""
    M, N = XO.shape
    one = torch.ones(N, dtype=torch.float64)
    zero = torch.zeros(M, N, dtype=torch.float64)
    dY = zero if dY is None else dY.double()
    dXO = zero if dXO is None else dXO.double()
    xhat, rx, magx = norm64(pre, XO.double(), eps)
    g = dY * (one if wpre is None else wpre.double())
    j, tj = jacobian(pre, xhat, rx, magx, g, zero)
    d = dXO + j
    td = tj + C32 * (dXO.abs() + j.abs())
    out = {"dX": (d, td)}
    nsum = (M + 64) * U32

    def col(v, t):
        return v.sum(0), t.sum(0) + (nsum + C32) * v.abs().sum(0) + 1e-30
    out["dpre_weight"] = col(dY * xhat, C32 * dY.abs() * magx)
    out["dpre_bias"] = col(dY, zero)
    if Z is None:
        return out
    zhat, rz, magz = norm64(post, Z.double(), eps)
    w = one if wpost is None else wpost.double()
    b = 0 * one if bpost is None else bpost.double()
    G = 0 if gate is None else gate.shape[0]
    gt = scale * (torch.ones(M, N, dtype=torch.float64) if gate is None
                  else gate.double().repeat_interleave(gate_rows, 0)[:M])
    dn, tn = gt * d, gt.abs() * (td + C32 * d.abs())
    out["dZ"] = jacobian(post, zhat, rz, magz, dn * w, (tn + C32 * dn.abs()) * w.abs())
    out["dpost_weight"] = col(dn * zhat, tn * magz + C32 * dn.abs() * magz)
    out["dpost_bias"] = col(dn, tn)
    if gate is not None:
        n = zhat * w + b
        v = scale * d * n
        # the kernel sums d zhat and d apart and joins them: their magnitudes count
        mag = abs(scale) * d.abs() * (magz * w.abs() + b.abs())
        t = abs(scale) * td * (magz * w.abs() + b.abs()) + (C32 + nsum) * mag
        idx = torch.arange(M) // gate_rows
        out["dgate"] = (torch.zeros(G, N, dtype=torch.float64).index_add_(0, idx, v),
                        torch.zeros(G, N, dtype=torch.float64).index_add_(0, idx, t) + 1e-30)
    return out
