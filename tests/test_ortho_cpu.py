"""The orthogonalised update on the CPU: exports, workspace and refusals (no GPU)."""
import mixed_precision_dense_sm_gb300 as lib


def test_declared():
    names = lib.declared_symbols()
    for n in ("ortho_update", "ortho_workspace"):
        assert n in names and hasattr(lib.lib, n)
    text = open(next(h for h in lib.HEADERS if "ortho" in h)).read()
    assert f"#define ORTHO_MAX_STEPS {lib.ORTHO_MAX_STEPS}\n" in text
    assert f"#define ORTHO_MAX_SIDE {lib.ORTHO_MAX_SIDE}\n" in text


def test_workspace():
    """X twice, A and B in 16 bits and X's low part in 8 on sides padded to 64; the same
    for a matrix and its transpose."""
    assert lib.ortho_workspace(0, 5, 5) == lib.ortho_workspace(2, 0, 5) == lib.ortho_workspace(2, 5, 0) == 0
    for bad in ((-1, 4, 4), (1, -4, 4), (1, 4, -4), (65536, 4, 4), (1, 65537, 4), (1, 4, 65537)):
        assert lib.ortho_workspace(*bad) == -1
    for batch, r, c in ((1, 1, 1), (3, 64, 100), (16, 1023, 777), (1, 4096, 14336), (65535, 65536, 65536)):
        n, m = (-(-v // 64) * 64 for v in sorted((r, c)))
        least = batch * (5 * n * m + 4 * n * n)
        got = lib.ortho_workspace(batch, r, c)
        assert got == lib.ortho_workspace(batch, c, r)
        assert least <= got <= least + 8192 + 8 * batch * n + 16384 * batch


def test_needs_a_handle():
    assert lib.ortho_update(None, 1, 8, 8, 256, 8, 0, lib.GEMM_F32, 256, 8, 0, (1.5, -0.5, 0.0)) == 1
