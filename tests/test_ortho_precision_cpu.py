"""The precision of the orthogonalised update by the model of its roundings (ortho_model):
what the header promises holds for it, and the check of the GPU tests sees a coarser
X, A or B and a wrong coefficient (mistakes planted in the model)."""
import pytest
import torch

import ortho_model as om
import ortho_ref as ortho


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("kind", om.KINDS)
def test_promise(kind, steps):
    """In the 2-norm, before FP32's errors; rank 1 and 4 below 0.001 at both."""
    G = om.update(kind, 128, 512)
    want, near = ortho.define(G, om.MUON, steps=steps), om.model(G, steps=steps)
    off = float((near - want).norm() / want.norm())
    assert off <= (0.001 if kind.startswith("rank") else om.PROMISE[steps]), off


def test_fine_steps():
    """The usual five steps enlarge by 484: none; each step more is one; Newton's 1.5 need 16."""
    assert [om.fine_steps([om.MUON] * n) for n in (1, 2, 5, 6, 8, 12)] == [0, 0, 0, 1, 3, 7]
    assert [om.fine_steps([(1.5, -0.5, 0.0)] * n) for n in (8, 15, 16, 32)] == [0, 0, 1, 17]
    assert om.fine_steps([(600.0, 0.0, 0.0)] * 2) == 1 and om.fine_steps([(600.0, 0.0, 0.0)]) == 0
    assert om.fine_steps([(0.1, 0.0, 0.0)] * 3 + [om.MUON] * 6) == 4


def test_late_step():
    assert [om.late_step([om.MUON] * n) for n in (1, 2, 3, 5, 8)] == [0, 0, 1, 3, 6]
    assert om.late_step([(1.5, -0.5, 0.0)] * 9) == 5 and om.late_step([(0.5, 0.0, 0.0)] * 9) == 0
    assert om.late_step([om.MUON] * 3 + [(5.0, 0.0, 0.0)]) == 3


def planted(kind, G, steps):
    X = ortho.wide(G.double())
    X = X / (X.norm() + 1e-7)
    a, b, c = om.MUON
    b *= 1.002 if kind == "b" else 1.0
    r16 = om.bf16 if kind == "bf16" else om.half
    for _ in range(steps):
        hi = r16(X)
        lo = X - hi
        if kind in ("no lo", "fp16", "bf16"):
            lo = torch.zeros_like(lo)
        elif kind in ("e5m2", "d lo"):
            lo = (lo * (om.SCALE * 1024)).float().to(torch.float8_e5m2).double() / (om.SCALE * 1024)
        else:
            lo = om.byte(lo, hi, om.PARTS * 256)
        A = hi @ hi.mT
        D = A.diagonal().clone() if kind not in ("fp16", "bf16") else torch.zeros(A.shape[0], dtype=torch.float64)
        A = r16(A - torch.diag(D)) + torch.diag(D)
        B = b * A + c * (A @ A)
        d = B.diagonal().clone() if kind not in ("fp16", "bf16") else D
        X = a * (hi + lo) + d[:, None] * (hi + (lo if kind == "d lo" else 0.0)) + r16(B - torch.diag(d)) @ hi
    return X


# Where each is seen.  (After eight steps noise is as exact without lo: a lo without B lo
# beside it is no gain there.  b off by 0.2 % weighs less than FP32's errors at rank 1 after eight steps.)
LOW = ("rank1", "rank4")
NOT_NOISE = tuple(k for k in om.KINDS if k != "noise")
CAUGHT = {
    "no lo": {5: om.KINDS, 8: NOT_NOISE},
    "fp16": {5: om.KINDS, 8: om.KINDS},
    "bf16": {5: om.KINDS, 8: om.KINDS},
    "b": {5: om.KINDS, 8: om.KINDS[1:]},
    "e5m2": {5: LOW + ("noise", "few", "decay6"), 8: LOW + ("decay4", "decay6")},
    "d lo": {5: LOW + ("noise", "decay4", "decay6"), 8: LOW + ("decay4", "decay6")},
}


@pytest.mark.parametrize("kind", om.KINDS)
@pytest.mark.parametrize("steps", [5, 8])
def test_the_check_sees(kind, steps):
    G = om.update(kind, 128, 512)
    om.check(om.model(G, steps=steps).float().bfloat16(), G, steps=steps)
    for mistake, where in CAUGHT.items():
        if kind in where[steps]:
            with pytest.raises(AssertionError):
                om.check(planted(mistake, G, steps).float().bfloat16(), G, steps=steps)
                raise RuntimeError(f"not seen: {mistake}")
