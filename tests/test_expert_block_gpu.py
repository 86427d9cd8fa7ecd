"""A feed-forward block with experts, as a training step and a decode step use it:
choices sorted, rows to their experts (expert_gather), each expert's gated layer and
down projection on its rows, rows back with the router's weights (expert_combine);
backward through all of it, clipping, and the orthogonalised updates of the experts'
weights.  The result is compared with the 64-bit composition of the same
definitions, with each stored tensor rounded where the step stores it."""
import math

import pytest
import torch

import expert_ref as ex
import ffn_ref as ref
import ortho_ref as ortho

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


class Experts:
    """y = sum over j of w_j Wd_e (silu(x Wg_e^T) * (x Wu_e^T)), e = ids_j, j = 0 .. k - 1."""

    def __init__(self, lib, tokens, k, experts, hidden, inner, drop, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.lib, self.g, self.E, self.F = lib, lib.Gemm(), experts, inner

        def w(*shape, scale=1.0, dt=BF):
            return (torch.randn(*shape, generator=gen) * scale).to(dt).cuda()
        logits = torch.randn(tokens, experts, generator=gen)
        top, ids = logits.topk(k, dim=1)
        ids[torch.rand(tokens, generator=gen) < drop] = -1
        self.ids, self.w = ids.cuda(), torch.softmax(top, 1).cuda()
        self.x, self.dy = w(tokens, hidden), w(tokens, hidden, scale=0.1)
        self.W = w(experts, 2 * inner, hidden, scale=hidden ** -0.5)
        self.Wd = w(experts, hidden, inner, scale=inner ** -0.5)
        rows = tokens * k
        z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")          # noqa: E731
        self.xs, self.zs, self.dzs, self.dxs = (z(rows, hidden) for _ in range(4))
        self.h, self.dh, self.P, self.dP = z(rows, inner), z(rows, inner), z(rows, 2 * inner), z(rows, 2 * inner)
        self.dW, self.dWd = torch.zeros_like(self.W), torch.zeros_like(self.Wd)
        self.dx, self.dw = torch.empty_like(self.x), torch.empty_like(self.w)

    def spans(self):
        o = self.offsets.tolist()
        return [(e, slice(o[e], o[e + 1])) for e in range(self.E) if o[e + 1] > o[e]]

    def forward(self):
        lib, g = self.lib, self.g
        self.pos, self.offsets, _ = lib.expert_sort(self.ids, self.E)
        lib.expert_gather(self.x, self.pos, Xs=self.xs)
        for e, r in self.spans():
            g.glu(self.xs[r], self.W[e], self.h[r], act="silu", P=self.P[r])
            g(self.h[r], self.Wd[e], self.zs[r], "N", "T")
        self.y = lib.expert_combine(self.zs, self.pos, self.w)

    def backward(self):
        lib, g = self.lib, self.g
        lib.expert_combine_backward(self.dy, self.pos, self.w, self.zs, dYs=self.dzs, dweight=self.dw)
        for e, r in self.spans():
            g(self.dzs[r], self.Wd[e], self.dh[r], "N", "N")
            g(self.dzs[r], self.h[r], self.dWd[e], "T", "N")
            g.glu_backward(self.dh[r], self.P[r], self.xs[r], self.W[e], act="silu", dP=self.dP[r], dX=self.dxs[r],
                           dW=self.dW[e])
        lib.expert_gather_backward(self.dxs, self.pos, dX=self.dx)

    def reference(self):
        d = lambda t: t.cpu().double()          # noqa: E731
        r = lambda t: t.to(BF).double()         # noqa: E731
        ids, w, x, W, Wd, F = self.ids.cpu(), d(self.w), d(self.x), d(self.W), d(self.Wd), self.F
        T, k = ids.shape
        pos, offsets, _ = ex.sort(ids, self.E)
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        dw, dW, dWd = torch.zeros_like(w), torch.zeros_like(W), torch.zeros_like(Wd)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not len(t):
                continue
            P = x[t] @ W[e].t()
            a = ref.act64("silu", P[:, :F])[0]
            h, P = r(a * P[:, F:]), r(P)
            z = r(h @ Wd[e].t())
            y.index_add_(0, t, z * w[t, j][:, None])
            dy = d(self.dy)[t]
            dw[t, j] = (dy * z).sum(1)
            dz = r(dy * w[t, j][:, None])
            dWd[e] = dz.t() @ h
            dP = r(ref.glu_backward(r(dz @ Wd[e]), P, x[t], W[e], "silu", BF, BF, BF)["dP"][0])
            dW[e] = dP.t() @ x[t]
            dx.index_add_(0, t, r(dP @ W[e]))
        return {"y": y, "dw": dw, "dW": dW, "dWd": dWd, "dx": dx}, pos, offsets


@pytest.mark.parametrize("tokens,k,experts,hidden,inner,drop", [
    (96, 2, 4, 256, 320, 0.0), (300, 3, 7, 200, 136, 0.2), (50, 4, 60, 129, 77, 0.3), (1, 2, 8, 256, 128, 0.0),
    (2500, 8, 16, 512, 256, 0.1)])
def test_training_step(lib, tokens, k, experts, hidden, inner, drop):
    """Each stored bf16 tensor is within half a step of the exact one, or one step off
    it where the two sides round apart; along the chain (six stored tensors) that
    stays below 6 steps, 6 * 2^-8 of the tensor's size, in the 2-norm."""
    b = Experts(lib, tokens, k, experts, hidden, inner, drop)
    b.forward()
    b.backward()
    b.g.sync()
    want, pos, offsets = b.reference()
    assert torch.equal(b.pos.cpu(), pos) and torch.equal(b.offsets.cpu(), offsets)
    for n, v in want.items():
        off = float((getattr(b, n).cpu().double() - v).norm() / v.norm().clamp_min(1e-30))
        assert off < 6 * 2.0 ** -8, (n, off)
    # the update: clipped by the global norm, then each expert's matrices
    total = math.sqrt(sum(float(want[n].square().sum()) for n in ("dW", "dWd")))
    norm = lib.grad_clip([b.dW, b.dWd], 0.5 * total)
    assert abs(float(norm) - total) < 6 * 2.0 ** -8 * total
    for grad in (b.dW, b.dWd):
        O = b.g.orthogonalize(grad, scale=0.2)
        b.g.sync()
        for e in sorted({0, experts // 2, experts - 1}):
            if grad[e].any():
                ortho.check(O[e], grad[e], MUON, scale=0.2)
            else:
                assert not O[e].any()
    b.g.close()


def test_decode_agrees_with_the_batch(lib):
    """Single tokens give what the same tokens gave in a batch, to the roundings of
    the tensors in between (four stored tensors: 4 steps)."""
    b = Experts(lib, 64, 4, 16, 512, 256, 0.0)
    b.forward()
    for i in (0, 31, 63):
        one = Experts(lib, 1, 4, 16, 512, 256, 0.0)
        one.W, one.Wd, one.x, one.ids, one.w = b.W, b.Wd, b.x[i:i + 1], b.ids[i:i + 1], b.w[i:i + 1]
        one.forward()
        off = float((one.y.double() - b.y[i:i + 1].double()).norm() / b.y[i].double().norm())
        assert off < 4 * 2.0 ** -8
        one.g.close()
    b.g.close()
