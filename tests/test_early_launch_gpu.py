"""Chains of operators in which each reads what the one before it just wrote,
into the same buffers over and over: back to back they give the bits that they
give with a wait for the GPU after every call."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def randn(gen, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def compare(start, step):
    """The outputs of step(wait) after runs from the same start, waiting or not."""
    def run(wait):
        state = {k: t.clone() for k, t in start.items()}
        torch.cuda.synchronize()
        for i in range(60):
            step(state, i, torch.cuda.synchronize if wait else lambda: None)
        torch.cuda.synchronize()
        return state
    a, b = run(True), run(False)
    for k in a:
        assert torch.isfinite(a[k].float()).all(), k
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("tokens,N,F", [(1, 512, 1024), (2, 1000, 520), (1, 4096, 4096), (8, 512, 1024)])
def test_decode_chain(tokens, N, F):
    """The norm writes the layer's input, the layer the product's, the product
    the norm's; the norm's weights are written by the clipping before it."""
    import mixed_precision_dense_sm_gb300 as lib
    gen = torch.Generator().manual_seed(tokens + N + F)
    W, Wd = randn(gen, 2 * F, N, scale=N ** -0.5), randn(gen, N, F, scale=F ** -0.5)
    src = [randn(gen, N, dtype=torch.float32) for _ in range(3)]
    bias = randn(gen, 2 * F, dtype=torch.float32)
    start = {"X": randn(gen, tokens, N), "Z": randn(gen, tokens, N), "Y": randn(gen, tokens, N),
             "H": randn(gen, tokens, F), "w": torch.ones(N, device="cuda"), "b": bias.clone()}
    g = lib.Gemm()
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(lib.grad_clip_workspace(2), dtype=torch.uint8, device="cuda")

    def step(s, i, wait):
        lib.grad_clip([src[i % 3], bias], 3.0 + i % 5, outputs=[s["w"], s["b"]], norm=norm, workspace=ws)
        wait()
        lib.norm_block(s["X"], s["Z"], s["X"], s["Y"], post="rms", post_weight=s["w"], pre="rms",
                       pre_weight=s["w"], scale=0.5)
        wait()
        g.glu(s["Y"], W, s["H"], bias=s["b"])
        wait()
        g(s["H"], Wd, s["Z"], transB="T")
        wait()
    compare(start, step)
    g.close()


@pytest.mark.parametrize("M,K,F", [(64, 256, 512), (100, 129, 65)])
def test_training_chain(M, K, F):
    """The backward passes' sums go through workspaces that every step writes again."""
    import mixed_precision_dense_sm_gb300 as lib
    gen = torch.Generator().manual_seed(M)
    W = randn(gen, 2 * F, K, scale=K ** -0.5)
    start = {"X": randn(gen, M, K), "Z": randn(gen, M, K), "Y": randn(gen, M, K), "H": randn(gen, M, F),
             "P": randn(gen, M, 2 * F), "dX": randn(gen, M, K), "g": randn(gen, M, K), "dZ": randn(gen, M, K),
             "dW": randn(gen, 2 * F, K), "db": randn(gen, 2 * F, dtype=torch.float32),
             "w": torch.ones(K, device="cuda"), "dw": torch.ones(K, device="cuda")}
    g = lib.Gemm()
    ws = torch.empty(lib.norm_block_backward_workspace(M, K), dtype=torch.uint8, device="cuda")
    cws = torch.empty(lib.grad_clip_workspace(2), dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")

    def step(s, i, wait):
        lib.norm_block(s["X"], s["Z"], s["X"], s["Y"], post="layer", pre="rms", pre_weight=s["w"], scale=0.25)
        wait()
        g.glu(s["Y"], W, s["H"], bias=s["db"], P=s["P"])
        wait()
        g.glu_backward(s["H"], s["P"], s["Y"], W, dP=s["P"], dX=s["dX"], dW=s["dW"], dbias=s["db"])
        wait()
        lib.norm_block_backward(s["X"], s["dX"], s["X"], s["Z"], pre="rms", pre_weight=s["w"], post="layer",
                                scale=0.25, dX=s["g"], dZ=s["dZ"], dpre_weight=s["dw"], workspace=ws)
        wait()
        lib.grad_clip([s["dw"], s["db"]], 1.0, outputs=[s["w"], s["db"]], norm=norm, workspace=cws)
        wait()
    compare(start, step)
    g.close()


@pytest.mark.parametrize("rows,cols", [(64, 1000), (300, 1023), (40, 33), (8, 70001), (4, 300000)])
@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "fp32"])
def test_softmax_after_the_kernel_that_writes_its_rows(rows, cols, dt):
    """Rows that clipping or a norm has just written, in place and apart."""
    import mixed_precision_dense_sm_gb300 as lib
    gen = torch.Generator().manual_seed(cols)
    src = [randn(gen, rows, cols, scale=2.0, dtype=dt) for _ in range(3)]
    start = {"X": randn(gen, rows, cols, dtype=dt), "Y": randn(gen, rows, cols, dtype=dt)}
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(lib.grad_clip_workspace(1), dtype=torch.uint8, device="cuda")
    small = cols <= lib.NORM_MAX_N

    def step(s, i, wait):
        lib.grad_clip([src[i % 3]], 10.0 + i % 7, outputs=[s["X"]], norm=norm, workspace=ws)
        wait()
        if small:
            lib.norm_block(s["X"], s["Y"], s["X"], pre=None, post="rms")
            wait()
        lib.softmax(s["X"], s["Y"])
        wait()
        lib.softmax(s["X"], s["X"])
        wait()
    compare(start, step)
