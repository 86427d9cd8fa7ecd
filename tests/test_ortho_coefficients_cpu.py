"""The orthogonalised update's coefficients are three for each step, or the call is
refused before anything else is looked at (no GPU)."""
import pytest

import mixed_precision_dense_sm_gb300 as lib

ABC = (1.5, -0.5, 0.0)


@pytest.mark.parametrize("n", [1, 2, 4, 5, 8])
def test_raw_call(n):
    with pytest.raises(ValueError):
        lib.ortho_update(None, 1, 8, 8, 256, 8, 0, lib.GEMM_F32, 256, 8, 0, (ABC * 3)[:n])


def test_raw_call_of_whole_steps():
    for n in (0, 1, 3):
        assert lib.ortho_update(None, 1, 8, 8, 256, 8, 0, lib.GEMM_F32, 256, 8, 0, ABC * n) == 1      # (no handle)


@pytest.fixture
def no_device(monkeypatch):
    if lib.torch is None:
        lib._need_torch()
    monkeypatch.setattr(lib, "_device", lambda t, name: -1)
    return monkeypatch


class Handle(lib.Gemm):
    """A Gemm without a device."""

    def __init__(self):
        self.h = None

    def __del__(self):
        pass


@pytest.mark.parametrize("steps,coefficients", [
    (3, ((1.5, -0.5),) * 3), (2, ((1.5, -0.5),) * 2), (3, ((1.5, -0.5, 0.0, 1.0),) * 3), (3, (ABC, ABC, (1.5, -0.5))),
    (3, (ABC, (1.5, -0.5), (1.5, -0.5, 0.0, 0.0))), (2, (ABC,)), (1, (ABC,) * 3), (5, (1.5, -0.5)), (4, ABC + ABC[:1])])
def test_method(no_device, steps, coefficients):
    G = lib.torch.zeros(4, 8)
    with pytest.raises(ValueError, match="coefficients"):
        Handle().orthogonalize(G, G.bfloat16(), steps=steps, coefficients=coefficients, stream=0)


def test_method_accepts_one_for_all_and_one_for_each(no_device):
    import numpy as np
    torch, seen = lib.torch, []
    G = torch.zeros(4, 8)
    no_device.setattr(lib, "ortho_update", lambda *a: seen.append(list(a[11])) or 0)
    for steps, c in ((3, ABC), (3, list(ABC)), (3, (ABC,) * 3), (3, np.array([ABC] * 3)), (3, torch.tensor([ABC] * 3))):
        Handle().orthogonalize(G, G.bfloat16(), steps=steps, coefficients=c, stream=0)
        assert [float(v) for v in seen[-1]] == list(ABC) * 3
