"""How exact the orthogonalised update is before its result is rounded to BF16: a model
of the kernels' roundings in 64 bits, and a check that sees a tenth of BF16's rounding.

Roundings: X is hi + lo, FP16 (times 2^11) and a byte of 254 parts to a step of hi, two
bytes (254 * 256 parts) before the first `fine` steps; A and B but for their diagonals
FP16.  X' = a (hi + lo) + d hi + (B - d) hi, from step `late` on with d lo as well.

Beside them the kernels have FP32's errors, small themselves, but what a rounding does to
a number next to its border they change altogether, and what the steps enlarge they
enlarge too.  How far apart that sets two runs is found by disturbing the model's sums
as FP32 does.  A tensor core aligns the products of an instruction and the sum so far to
the largest of them and cuts them off behind 24 bits (Fasi, Higham, Mikaitis and Pranesh,
Numerical behavior of NVIDIA tensor cores, 2021): K products are cut off, each by up to
2^-23 of a binade that is up to twice the sum, evenly, so by 2 * 2^-23 / sqrt(12) usually,
and all of them by sqrt(K) times that, sqrt(K) 2^-23.8 of a sum that is the sum of the
magnitudes at most: sqrt(K) 2^-24 of the latter are taken.  What is cut off is cut off
towards zero, so where the products have one sign it adds up: up to K times half of 2^-23 of
the sum so far, which is half the sum usually, in a binade of up to twice that: K 2^-24 of
the sum at most (a side of 65536: 2^-8; A of one column: 2^-11 in eight parts of K, seen),
of which each product of a run takes a part between none and all.  (2^-21 for any K, as if only
sums were cut off, is a sixth of it at K = 2048 and falls short.)  X' is disturbed by 2^-24,
the factor of G by 2^-22 (the norm's FP32 part, the quotient, the product) and each of its
products by a rounding.  A disturbed run stands for the kernels': its distance
from the definition and from the undisturbed model, means over the elements, are allowed
with a quarter more (three such runs agree to a tenth where roundings rule; where FP32's
errors do, the disturbance is larger than they are).

O is a rounding of something close to the model's: a number that is off by e before the
rounding lands on the neighbour with a chance of |e| over a step, so the mean of
|O - bf16(model)| is the mean of |e|."""
import torch

import ffn_ref as ref
import ortho_ref as ortho

MUON = (3.4445, -4.7750, 2.0315)
SCALE, PARTS, FINE_FROM, LATE_FROM = 2048.0, 254, 512.0, 4.0


def steps_of(coefficients, steps):
    return list(coefficients) if hasattr(coefficients[0], "__len__") else [coefficients] * steps


def fine_steps(abc):
    """The first steps: those that enlarge, with those behind them, by more than FINE_FROM."""
    n = len(abc) - 1
    grow = max(1.0, abs(abc[n][0]))
    while n > 0:
        grow *= max(1.0, abs(abc[n - 1][0]))
        if grow > FINE_FROM:
            break
        n -= 1
    return n


def late_step(abc):
    """The first of the last steps, behind each of which a rounding is enlarged by up to
    LATE_FROM."""
    s, grow = len(abc) - 1, 1.0
    while s > 0:
        grow *= max(1.0, abs(abc[s][0]))
        if grow > LATE_FROM:
            break
        s -= 1
    return s


def half(x):
    return (x * SCALE).float().half().double() / SCALE


def byte(lo, hi, parts):
    """lo in whole parts of a step of hi."""
    e = torch.frexp((hi * SCALE).float())[1].double() - 1
    step = torch.exp2(torch.where(hi == 0, -14.0, e).clamp(min=-14.0) - 10) / SCALE
    return torch.round(lo / step * parts) * step / parts


def parts_of(s, fine):
    return PARTS * 256 if s < fine else PARTS


def model(G, coefficients=MUON, eps=1e-7, scale=1.0, steps=5, gen=None):
    """scale * X with the kernels' roundings; gen: a generator of disturbances."""
    abc = steps_of(coefficients, steps)
    fine, late = fine_steps(abc), late_step(abc)
    X = ortho.wide(G.double())
    X = X / (X.norm() + eps)

    def rand(shape):
        return torch.randn(shape, generator=gen, dtype=torch.float64).to(X.device)

    def off(x, y, symmetric=True):
        if gen is None:
            return 0.0
        magnitudes = x.abs() @ y.abs()
        k = x.shape[1]
        n = k ** 0.5 * 2.0 ** -24 * rand(magnitudes.shape) * magnitudes
        cut = k * 2.0 ** -24 * float(torch.rand(1, generator=gen)) * (x @ y)
        return ((n + n.mT) / 2 ** 0.5 if symmetric else n) - cut

    if gen is not None:
        X = (X * (1 + 2.0 ** -22 * float(rand((1,))))).float().double()
    for s, (a, b, c) in enumerate(abc):
        hi = half(X)
        lo = byte(X - hi, hi, parts_of(s, fine))
        A = hi @ hi.mT + off(hi, hi.mT)
        D = A.diagonal().clone()
        A = half(A - torch.diag(D))
        A.diagonal().zero_()
        B = b * (A + torch.diag(D)) + c * (A @ A + D[:, None] * A + A * D + torch.diag(D * D))
        if gen is not None:
            B = B + c * off(A, A)
        d = B.diagonal().clone()
        B = half(B - torch.diag(d))
        X = a * (hi + lo) + d[:, None] * (hi + lo if s >= late else hi) + B @ hi + off(B, hi, False)
        if gen is not None:
            X = X * (1 + 2.0 ** -24 * rand(X.shape))
    X = scale * X
    return X.mT if G.shape[0] > G.shape[1] else X


def largest(G, coefficients, eps, steps):
    """Each element's largest magnitude before any step or behind the last, over the
    matrix's usual one there."""
    X = ortho.wide(G.double())
    X = X / (X.norm() + eps)
    most = torch.zeros_like(X)
    for a, b, c in steps_of(coefficients, steps) + [(0.0, 0.0, 0.0)]:
        most = torch.maximum(most, X.abs() / X.square().mean().sqrt())
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return most.mT if G.shape[0] > G.shape[1] else most


def apart(x, y, want):
    return float((x - y).abs().sum() / want.abs().sum())


def bf16(x):
    return x.float().bfloat16().double()


def figures(O, G, coefficients=MUON, eps=1e-7, scale=1.0, steps=5):
    """Mean magnitudes before the rounding, over the definition's: O off the definition,
    at most a disturbed run is, O off the model, at most a disturbed run is; and (model,
    the latter in the 2-norm per element)."""
    want = ortho.define(G, coefficients, eps, scale, steps)
    near = model(G, coefficients, eps, scale, steps)
    runs = [model(G, coefficients, eps, scale, steps, torch.Generator().manual_seed(i)) for i in range(3)]
    got = O.double()
    return (apart(got, bf16(want), want), max(apart(o, want, want) for o in runs),
            apart(got, bf16(near), want), max(apart(o, near, want) for o in runs)), \
        (near, max(float((o - near).square().mean().sqrt()) for o in runs))


def check(O, G, coefficients=MUON, eps=1e-7, scale=1.0, steps=5, most=None):
    """One matrix of 40000 elements or more.  The means are over the few that land on a
    neighbour, n of them with a standard deviation of sqrt(n), each off by a step of up to
    2^-6 of the mean magnitude (2^-7 of its own): six of these deviations more, and six
    such steps.  `most`: what the mean error before the rounding may be."""
    assert O.dtype == torch.bfloat16 and O.shape == G.shape and O.numel() >= 40000
    (off, run_off, near_off, run_near), (near, rms) = figures(O, G, coefficients, eps, scale, steps)
    step = 2.0 ** -6 / O.numel()

    def allowed(mean):
        return 1.25 * mean + 6 * (mean * step) ** 0.5 + 6 * step

    assert off <= allowed(run_off), f"off by {off:.5f}, disturbed runs by {run_off:.5f}"
    assert near_off <= allowed(run_near), f"off the model by {near_off:.5f}, disturbed runs by {run_near:.5f}"
    assert most is None or off <= most, f"off by {off:.5f}, at most {most}"
    # Each element: six times the usual distance (of a million elements the largest is at
    # 4.9 sigma), in proportion to its size.  Its size is the largest that it had on the
    # way: hi's rounding is half a step of X before each step, so up to 2^-11 |X|, and a
    # times it, or d times it, is part of the result, which may be small itself (an
    # update of rank 1 but for its own rounding to BF16 starts with an element at 4.4
    # times the usual and ends with it at 0.2).
    e = 6 * 1.25 * rms * (1 + largest(G, coefficients, eps, steps))
    ref.check(O, near.cpu(), (e + ref.rounding(near.abs() + e, torch.bfloat16)).cpu(), "O")
    return off


def update(kind, r, c, seed=0, dtype=torch.float32):
    """rankN; noise; few (n / 32 strong directions over noise); decayN: singular values
    from 1 to 10^-N, even in the logarithm."""
    gen = torch.Generator().manual_seed(seed + 3 * r + c)
    n = min(r, c)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    if kind.startswith("rank"):
        k = int(kind[4:])
        G = randn(r, k) @ randn(k, c)
    elif kind == "noise":
        G = randn(r, c)
    elif kind == "few":
        k = max(1, n // 32)
        G = 0.3 * randn(r, c) + randn(r, k) @ randn(k, c)
    else:
        u, v = torch.linalg.qr(randn(r, n))[0], torch.linalg.qr(randn(c, n))[0]
        G = (u * torch.logspace(0, -float(kind[5:]), n)) @ v.T
    return G.to(dtype)


# What the header promises: the mean error before the rounding to BF16, of the usual
# coefficients.  (Low rank after eight steps: FP32's own errors, enlarged.)
PROMISE = {5: 0.0015, 8: 0.003}
KINDS = ("rank1", "rank4", "noise", "few", "decay2", "decay4", "decay6")
