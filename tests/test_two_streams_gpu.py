"""Calls that overlap on the GPU: two streams, each with its own handle and
workspaces, give the bits that each gives alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Work:
    """One stream's operators and tensors.  (No tile schedule here waits for other
    CTAs of its grid but for those of its own cluster.)"""

    def __init__(self, lib, seed, M, N, F):
        gen = torch.Generator().manual_seed(seed)

        def randn(*shape, scale=1.0, dtype=BF):
            return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()
        self.lib, self.g, self.args = lib, lib.Gemm(), (M, N, F)
        self.X, self.Z, self.dY = randn(M, N), randn(M, N), randn(M, N)
        self.w, self.gate = randn(N, dtype=torch.float32), randn(-(-M // 5), N, dtype=torch.float32)
        self.T, self.W = randn(16, N), randn(2 * F, N, scale=N ** -0.5)
        self.out = {}
        self.new = {"XO": (M, N), "Y": (M, N), "dX": (M, N), "dZ": (M, N), "H1": (1, F), "H2": (2, F), "H16": (16, F)}

    def run(self, stream):
        lib, (M, N, F) = self.lib, self.args
        o = {k: torch.empty(s, dtype=BF, device="cuda") for k, s in self.new.items()}
        o.update({k: torch.empty(N, device="cuda") for k in ("dw", "db")})
        o["dgate"] = torch.empty_like(self.gate)
        o["norm"], o["clip"] = torch.empty(1, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
        ws = torch.empty(lib.norm_block_backward_workspace(M, N, 5), dtype=torch.uint8, device="cuda")
        cws = torch.empty(lib.grad_clip_workspace(1), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        kw = dict(pre="rms", pre_weight=self.w, post="layer", post_weight=self.w, gate=self.gate, gate_rows=5,
                  stream=stream)

        def step():
            lib.norm_block(self.X, self.Z, o["XO"], o["Y"], **kw)
            lib.norm_block_backward(o["XO"], self.dY, o["Y"], self.Z, dX=o["dX"], dZ=o["dZ"], dpre_weight=o["dw"],
                                    dpre_bias=o["db"], dgate=o["dgate"], workspace=ws, **kw)
            for m in (1, 2, 16):
                self.g.glu(self.T[:m], self.W, o[f"H{m}"], stream=stream)
            lib.grad_clip([o["dX"]], 1.0, outputs=[o["clip"]], norm=o["norm"], workspace=cws, stream=stream)
        return o, step, (ws, cws)


@pytest.mark.parametrize("a,b", [((700, 4096, 4096), (900, 1000, 2048)), ((200, 12288, 1024), (3000, 264, 4096))])
def test_two_streams(a, b):
    import mixed_precision_dense_sm_gb300 as lib
    works = [Work(lib, i, *s) for i, s in enumerate((a, b))]
    for (M, N, F) in (a, b):
        for m in (1, 2, 16):
            st, p = lib.glu_plan_query(m, F, N, 256, N, 256, N, 256, F, (lib.GEMM_BF16,) * 3)
            assert st == 0 and p["sk_len"] == 0 and p["path_name"] in ("dot", "skinny")
    alone = []
    for w in works:
        o, step, keep = w.run(0)
        step()
        torch.cuda.synchronize()
        alone.append(o)
    streams = [torch.cuda.Stream() for _ in works]
    runs = [w.run(s.cuda_stream) for w, s in zip(works, streams)]
    for _ in range(40):
        for _, step, _ in runs:
            step()
    torch.cuda.synchronize()
    for (o, _, _), want in zip(runs, alone):
        for k in want:
            assert torch.isfinite(want[k].float()).all() and torch.equal(o[k], want[k]), k
    for w in works:
        w.g.close()


@pytest.mark.parametrize("shapes", [((64, 14336, 4096), (64, 4096, 14336)), ((64, 16384, 8192), (3136, 512, 4608))])
def test_stream_k_on_two_streams(shapes):
    """Stream-K kernels of two streams share the SMs: a finisher waits only for
    blocks started before it, so every call ends, with the bits it has alone."""
    import mixed_precision_dense_sm_gb300 as lib
    runs = []
    for i, (M, N, K) in enumerate(shapes):
        gen = torch.Generator().manual_seed(i)
        st, p = lib.gemm_plan_query("N", "T", M, N, K, 1.0, 256, K, 256, K, 0.0, 256, N,
                                    (lib.GEMM_BF16, lib.GEMM_BF16, lib.GEMM_F32))
        assert st == 0 and p["sk_len"] > 0, p
        A, B = torch.randn(M, K, generator=gen).to(BF).cuda(), torch.randn(N, K, generator=gen).to(BF).cuda()
        C, h = torch.empty(M, N, device="cuda"), lib.Gemm()
        h(A, B, C, transB="T")
        h.sync()
        runs.append((h, A, B, C, C.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(100):
        for h, A, B, C, _, s in runs:
            h(A, B, C, transB="T", stream=s.cuda_stream)
    for h, A, B, C, want, s in runs:
        h.sync(s.cuda_stream)
        assert torch.equal(C, want)
        h.close()
