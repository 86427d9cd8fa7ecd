"""The gated layer's plans at the longest rows (no GPU)."""
import pytest

import mixed_precision_dense_sm_gb300 as lib

BF16 = lib.GEMM_BF16


@pytest.mark.parametrize("M", [1, 3, 64, 128, 200, 5000])
@pytest.mark.parametrize("pad", [0, 1])
def test_every_k_has_a_plan(M, pad):
    """Copies of unaligned rows are padded to pairs of K chunks, but not past the
    largest K."""
    for K in (*range(2 ** 31 - 130, 2 ** 31, 7), 2 ** 31 - 1):
        st, p = lib.glu_plan_query(M, 64, K, 256, K + pad, 256, K + pad, 256, 64, (BF16, BF16, BF16))
        assert st == 0, (K, st)
        if p["path_name"] != "dot":
            assert p["k_blocks"] * p["block_k"] >= K
