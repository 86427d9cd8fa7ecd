"""The feed-forward operators together, as a training step and a decode step
use them: norm, gated layer, down projection (gemm_run), norm with gate and
residual; backward through all of it, then the global norm and clipping.  The
result is compared with the 64-bit composition of the same definitions, with
each stored tensor rounded where the step stores it."""
import math

import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    import mixed_precision_dense_sm_gb300 as lib
    return lib


class Block:
    """x -> x + 0.5 * gate * RMSNorm(Wd (silu(n Wg^T) * (n Wu^T))), n = LayerNorm(x),
    and the norm of the next block."""

    def __init__(self, lib, tokens, hidden, inner, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.lib, self.g = lib, lib.Gemm()
        self.M, self.N, self.F = tokens, hidden, inner

        def w(*shape, scale=1.0, mean=0.0, dt=BF):
            return (torch.randn(*shape, generator=gen) * scale + mean).to(dt).cuda()
        self.x = w(tokens, hidden)
        self.W = w(2 * inner, hidden, scale=hidden ** -0.5)
        self.Wd = w(hidden, inner, scale=inner ** -0.5)
        self.w1, self.b1 = w(hidden, scale=0.1, mean=1.0, dt=F32), w(hidden, scale=0.1, dt=F32)
        self.wp, self.gate = w(hidden, scale=0.1, mean=1.0, dt=F32), w(1, hidden, scale=0.1, mean=0.5, dt=F32)
        self.w2 = w(hidden, scale=0.1, mean=1.0, dt=F32)
        self.dxo, self.dy = w(tokens, hidden, scale=0.1), w(tokens, hidden, scale=0.1)
        e = torch.empty
        self.n, self.h = e(tokens, hidden, dtype=BF, device="cuda"), e(tokens, inner, dtype=BF, device="cuda")
        self.P = e(tokens, 2 * inner, dtype=BF, device="cuda")
        self.z, self.xo, self.y = (torch.empty_like(self.x) for _ in range(3))
        self.dz, self.dn, self.dx = (torch.empty_like(self.x) for _ in range(3))
        self.dx2 = torch.empty_like(self.x)
        self.dh, self.dP = torch.empty_like(self.h), torch.empty_like(self.P)
        self.dW, self.dWd = torch.empty_like(self.W), torch.empty_like(self.Wd)
        self.dw1, self.db1, self.dwp, self.dw2 = (torch.empty_like(t) for t in (self.w1, self.b1, self.wp, self.w2))
        self.dgate = torch.empty_like(self.gate)

    def forward(self, save=True):
        lib, g = self.lib, self.g
        lib.norm_block(self.x, Y=self.n, pre="layer", pre_weight=self.w1, pre_bias=self.b1, eps=EPS)
        g.glu(self.n, self.W, self.h, act="silu", P=self.P if save else None)
        g(self.h, self.Wd, self.z, "N", "T")
        lib.norm_block(self.x, self.z, self.xo, self.y, pre="rms", pre_weight=self.w2, post="rms",
                       post_weight=self.wp, gate=self.gate, gate_rows=self.M, scale=0.5, eps=EPS)

    def backward(self):
        lib, g = self.lib, self.g
        # dx: the residual branch's part
        lib.norm_block_backward(self.xo, self.dy, self.dxo, self.z, pre="rms", pre_weight=self.w2,
                                post="rms", post_weight=self.wp, gate=self.gate, gate_rows=self.M,
                                scale=0.5, eps=EPS, dX=self.dx, dZ=self.dz, dgate=self.dgate,
                                dpre_weight=self.dw2, dpost_weight=self.dwp)
        g(self.dz, self.Wd, self.dh, "N", "N")
        g(self.dz, self.h, self.dWd, "T", "N")
        g.glu_backward(self.dh, self.P, self.n, self.W, act="silu", dP=self.dP, dX=self.dn, dW=self.dW)
        lib.norm_block_backward(self.x, self.dn, self.dx, pre="layer", pre_weight=self.w1, eps=EPS,
                                dX=self.dx2, dpre_weight=self.dw1, dpre_bias=self.db1)

    def grads(self):
        return [self.dW, self.dWd, self.dw1, self.db1, self.dwp, self.dgate, self.dw2]

    def reference(self):
        """The same step in 64 bits; stored tensors rounded as the step stores them."""
        d = lambda t: t.cpu().double()          # noqa: E731
        r = lambda t: t.to(BF).double()         # noqa: E731
        x, W, Wd, F = d(self.x), d(self.W), d(self.Wd), self.F
        n = r(ref.norm_pre(x, "layer", d(self.w1), d(self.b1), EPS)[0])
        P = n @ W.t()
        a, _, _, _ = ref.act64("silu", P[:, :F])
        h = r(a * P[:, F:])
        P = r(P)
        z = r(h @ Wd.t())
        xo = r(ref.norm_block(x, z, None, None, None, "rms", d(self.wp), None, d(self.gate), self.M, 0.5, EPS)[0])
        y = ref.norm_pre(xo, "rms", d(self.w2), None, EPS)[0]
        b = ref.norm_block_backward(xo, d(self.dy), d(self.dxo), z, "rms", d(self.w2), "rms", d(self.wp), None,
                                    d(self.gate), self.M, 0.5, EPS)
        dz, dx = r(b["dZ"][0]), r(b["dX"][0])
        dh = r(dz @ Wd)
        gb = ref.glu_backward(dh, P, n, W, "silu", BF, BF, BF)
        dP = r(gb["dP"][0])
        dn = r(dP @ W)
        c = ref.norm_block_backward(x, dn, dx, None, "layer", d(self.w1), None, None, None, None, 1, 1.0, EPS)
        return {"xo": xo, "y": y, "dx2": c["dX"][0], "dW": dP.t() @ n, "dWd": dz.t() @ h,
                "dw1": c["dpre_weight"][0], "db1": c["dpre_bias"][0], "dwp": b["dpost_weight"][0],
                "dgate": b["dgate"][0], "dw2": b["dpre_weight"][0]}


@pytest.mark.parametrize("tokens,hidden,inner", [(96, 256, 640), (257, 200, 300), (40, 129, 77), (1, 512, 1024),
                                                 (512, 1024, 2048)])
def test_training_step(lib, tokens, hidden, inner):
    """Each stored bf16 tensor is within half a step of the exact one, or one
    step off it where the two sides round apart; along the chain (six stored
    tensors) that stays below 6 steps, 6 * 2^-8 of the tensor's size, in the
    2-norm."""
    b = Block(lib, tokens, hidden, inner)
    b.forward()
    b.backward()
    want = b.reference()
    for k, v in want.items():
        got = getattr(b, k).cpu().double()
        off = float((got - v).norm() / v.norm().clamp_min(1e-30))
        assert off < 6 * 2.0 ** -8, (k, off)
    total = math.sqrt(sum(float((v * v).sum()) for k, v in want.items() if k in
                          ("dW", "dWd", "dw1", "db1", "dwp", "dgate", "dw2")))
    outs = [torch.empty_like(t) for t in b.grads()]
    norm = lib.grad_clip(b.grads(), 0.5 * total, outputs=outs)
    assert abs(float(norm) - total) < 6 * 2.0 ** -8 * total
    after = lib.grad_clip(outs, math.inf)
    # one rounding of each element on the way
    assert abs(float(after) - 0.5 * total) < 2.0 ** -8 * total
    b.g.close()


def test_decode_agrees_with_the_batch(lib):
    """Single tokens give what the same tokens gave in a batch, to the
    roundings of the tensors in between."""
    b = Block(lib, 64, 512, 1024)
    b.forward()
    xo, y = b.xo.clone(), b.y.clone()
    for i in (0, 7, 63):
        one = Block(lib, 1, 512, 1024)
        for k in ("W", "Wd", "w1", "b1", "wp", "gate", "w2"):
            setattr(one, k, getattr(b, k))           # the same model
        one.x.copy_(b.x[i:i + 1])
        one.forward(save=False)
        for got, want in ((one.xo, xo[i:i + 1]), (one.y, y[i:i + 1])):
            assert float((got.float() - want.float()).norm() / want.float().norm()) < 3 * 2.0 ** -8
        one.g.close()
    b.g.close()


def test_step_in_a_graph_beside_an_eager_one(lib):
    """The whole step captured, replayed while another block's step runs on
    another stream with its own handle, twice with the same bits."""
    a, e = Block(lib, 300, 256, 520, 1), Block(lib, 300, 256, 520, 2)

    def step(b):
        b.forward()
        b.backward()
        return lib.grad_clip(b.grads(), 1.0)
    for b in (a, e):
        step(b)
    torch.cuda.synchronize()
    want_e = [t.clone() for t in e.grads()]
    e_first = [t.clone() for t in (e.dx2, e.y)]
    a_first = [t.clone() for t in (a.dx2, a.y, *a.grads())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
        with torch.cuda.stream(s):
            step(e)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((a.dx2, a.y, *a.grads()), a_first))
        assert all(torch.equal(x, y) for x, y in zip((e.dx2, e.y), e_first))
        assert all(torch.equal(x, y) for x, y in zip(e.grads(), want_e))
        assert math.isfinite(float(norm))
    for b in (a, e):
        b.g.close()


def test_new_tensors_on_another_stream():
    """Tensors that a call on a given stream makes are not taken from memory
    that the current stream has freed and still writes to."""
    import mixed_precision_dense_sm_gb300 as lib
    g = lib.Gemm()
    gen = torch.Generator().manual_seed(8)
    X = torch.randn(256, 512, generator=gen).to(torch.bfloat16).cuda()
    W = torch.randn(1024, 512, generator=gen).to(torch.bfloat16).cuda()
    v = torch.ones(512, device="cuda")
    dv = torch.empty_like(v)

    def calls(stream):
        H = g.glu(X, W, stream=stream)
        XO, Y = lib.norm_block(X, H, post="rms", pre_weight=v, stream=stream)
        lib.norm_block_backward(XO, Y, Z=H, post="rms", pre_weight=v, dpre_weight=dv, stream=stream)
        return [H, XO, Y, dv.clone() if stream is None else dv, lib.grad_clip([H, XO], 1.0, outputs=outs, stream=stream)]
    outs = [torch.empty(256, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [t.clone() for t in calls(None)]
    dv.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                # the current stream is late
    tmp = [torch.empty(n, dtype=torch.uint8, device="cuda")
           for n in (4, 512, 4096, 1 << 18, 1 << 18, 1 << 18, 1 << 20, 1 << 20, 1 << 22)]
    for t in tmp:
        t.fill_(255)
    del tmp, t
    got = calls(side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g.close()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N", [1, 25, 1001, 1002, 1003, 2388, 2389])
def test_padding_behind_rows_of_odd_bytes(N, dt):
    """The columns between N and an aligned pitch stay as they were, and what
    lies behind a last row without padding, for the GEMM and the gated layer."""
    import mixed_precision_dense_sm_gb300 as lib
    g = lib.Gemm()
    ld = -(-N // 8) * 8
    for M, K in ((704, 3626), (5000, 2048), (20000, 64)):
        A = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        W = torch.randn(2 * N, K, device="cuda").to(torch.bfloat16)
        for f in (lambda C: g(A, W[:N], C, transB="T"), lambda C: g.glu(A, W, C)):
            buf = torch.full((M * ld + 16,), 321.0, dtype=dt, device="cuda")
            f(buf[:M * ld].view(M, ld)[:, :N])
            g.sync()
            assert (buf[:M * ld].view(M, ld)[:, N:] == 321).all() and (buf[M * ld:] == 321).all(), (M, K)
    g.close()
