"""The orthogonalised update in 64 bits: the definition, the definition with the
kernels' roundings to 16 bits, and the bounds its tests use.

Notation of one step: A = X X^T, B = b A + c A^2, X' = a X + B X, f(s) = a s + b s^3
+ c s^5 on the singular values s of X.

First-order bound, in Frobenius norms.  With u = 2^-11 (a rounding to FP16), 2^-14 for the
pair (half a step of hi, 2^-11, and of E5M2 of that, 2^-3) and t the
relative error of an FP32 sum of products of the tensor core (the products' tests
allow 1e-5 of the sum of magnitudes, at most ||X||_F^2 for A, ||A||_F^2 for A^2 and
||B||_F ||X||_F for B X):
    dA <= 2 u |X| ||X|| + u ||A|| + t ||X||^2             |.| the largest singular value
    dB <= (|b| + 2 |c| |A|) dA + t |c| ||A||^2 + u ||B||
    dX' <= |X| dB + u |B| ||X|| + t ||B|| ||X|| + 2^-14 ||X'||
(A's and B's diagonals are not rounded, and B's multiplies all of X: the bound holds as
it is.)
A change E of X reaches the end through the steps that are left, g = f(f(...)): in the
singular vectors' basis its parts are multiplied by (g(s) - g(s')) / (s - s') and
(g(s) + g(s')) / (s + s'), so by at most the largest of these."""
import torch

import ffn_ref as ref

U16, TC = 2.0 ** -11, 1e-5
SCALE = 2048.0


def wide(G):
    return G.mT if G.shape[-2] > G.shape[-1] else G


def define(G, coefficients, eps=1e-7, scale=1.0, steps=5):
    """scale * X after the steps, for one matrix."""
    abc = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    X = wide(G.double())
    X = X / (X.norm() + eps)
    for a, b, c in abc:
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    X = scale * X
    return X.mT if G.shape[-2] > G.shape[-1] else X


def _half(x):
    return (x * SCALE).float().half().double() / SCALE


def _low(x):
    return (x * (SCALE * 1024)).float().to(torch.float8_e5m2).double() / (SCALE * 1024)


def rounded(G, coefficients, eps=1e-7, scale=1.0, steps=5):
    """The same with the kernels' roundings: A and B but for their diagonals to FP16, X a
    pair of an FP16 and an E5M2 number, of which the first enters the products."""
    abc = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    X = wide(G.double())
    X = X / (X.norm() + eps)
    for i, (a, b, c) in enumerate(abc):
        hi = _half(X)
        X = hi + _low(X - hi)
        A = hi @ hi.mT
        d = A.diagonal().clone()
        A = _half(A - torch.diag(d)) + torch.diag(d)
        B = b * A + c * (A @ A)
        d = B.diagonal().clone()
        B.diagonal().zero_()
        X = (a + d)[:, None] * X + _half(B) @ hi
    X = scale * X
    return X.mT if G.shape[-2] > G.shape[-1] else X


def _growth(s, abc):
    """Most that the steps abc enlarge a change of a matrix of singular values s."""
    if not abc:
        return 1.0
    g, d = s.clone(), torch.ones_like(s)
    for a, b, c in abc:
        d = d * (a + 3 * b * g ** 2 + 5 * c * g ** 4)
        g = a * g + b * g ** 3 + c * g ** 5
    gap = s[:, None] - s[None]
    near = gap.abs() < 1e-7
    minus = torch.where(near, d[:, None].expand_as(gap), (g[:, None] - g[None]) / torch.where(near, 1.0, gap))
    both = s[:, None] + s[None]
    plus = torch.where(both > 1e-12, (g[:, None] + g[None]) / both.clamp(min=1e-12), d[:, None].expand_as(gap))
    return float(torch.maximum(minus.abs(), plus.abs()).max())


def bound(G, coefficients, eps=1e-7, scale=1.0, steps=5):
    """(Frobenius bound on O before its rounding, the same for FP16's roundings alone)."""
    abc = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    s = torch.linalg.svdvals(wide(G.double().cpu()))
    s = s / (s.norm() + eps)
    all_, half = 2.0 ** -14 * float(s.norm()) * _growth(s, abc), 0.0
    for i, (a, b, c) in enumerate(abc):
        A, B = s ** 2, b * s ** 2 + c * s ** 4
        new = a * s + B * s
        n = lambda v: float(v.norm())
        m = lambda v: float(v.abs().max())

        def local(u, t):
            dA = 2 * u * m(s) * n(s) + u * n(A) + t * n(s) ** 2
            dB = (abs(b) + 2 * abs(c) * m(A)) * dA + t * abs(c) * n(A) ** 2 + u * n(B)
            return m(s) * dB + u * m(B) * n(s) + t * n(B) * n(s) + 2.0 ** -14 * n(new)

        grow = _growth(new.abs(), abc[i + 1:])
        all_ += grow * local(U16, TC)
        half += grow * local(U16, 0.0)
        s = new.abs()
    return abs(scale) * all_, abs(scale) * half


def check(O, G, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, steps=5):
    """One matrix: O against the definition in norm; and elementwise against the
    definition with its roundings, where what differs is the rare entry of A or B that
    FP32's sums put on the other side of a rounding border: one in 32 at most, so a
    part sqrt(1/32) of the bound for all of them, spread over the elements, six
    sigma."""
    assert O.dtype == torch.bfloat16 and O.shape == G.shape
    got = O.cpu().double()
    want = define(G, coefficients, eps, scale, steps).cpu()
    full, half = bound(G, coefficients, eps, scale, steps)
    tol = full + float(ref.rounding(want, torch.bfloat16).norm())
    err = float((got - want).norm())
    assert err <= tol, f"norm of the error {err:.3g}, bound {tol:.3g}, norm {float(want.norm()):.3g}"
    near = rounded(G, coefficients, eps, scale, steps).cpu()
    e = 6 * (1 / 32) ** 0.5 * half / want.numel() ** 0.5
    ref.check(O, near, e + ref.rounding(near.abs() + e, torch.bfloat16), "O")
    return err / max(float(want.norm()), 1e-300)
