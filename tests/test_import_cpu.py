"""The package without torch: planning and the raw C calls need only the library."""
import os
import subprocess
import sys

import mixed_precision_dense_sm_gb300 as lib

WITHOUT = """
import sys
sys.modules["torch"] = None                      # importing it fails
import mixed_precision_dense_sm_gb300 as lib
bf, f32 = lib.GEMM_BF16, lib.GEMM_F32
assert lib.gemm_plan_query("N", "T", 64, 512, 256, 1.0, 256, 256, 256, 256, 0.0, 256, 512, (bf, bf, f32))[0] == 0
assert lib.glu_plan_query(64, 512, 256, 256, 256, 256, 256, 256, 512, (bf, bf, bf))[0] == 0
assert lib.softmax_plan_query(64, 512, 256, 512, f32, 256, 512, f32)[0] == 0
assert lib.glu_forward(None, 1, 1, 1, 256, 1, 256, 1, 256, 1, (bf, bf, bf)) == 1
assert lib.norm_block_backward_workspace(64, 512, 1, 152) > 0 and lib.grad_clip_workspace(3, 152) > 0
assert lib.grad_clip_raw([0], None, [4], [f32], 1.0, 1.0, 256, 256, 1 << 20) == 1
assert lib.declared_symbols()
"""

LAZY = """
import sys
import mixed_precision_dense_sm_gb300 as lib
assert "torch" not in sys.modules
import torch
assert lib.dtype_code(torch.bfloat16) == lib.GEMM_BF16
"""


def run(code):
    env = {k: v for k, v in os.environ.items() if not k.startswith("PYTEST")}
    out = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(lib.HERE), env=env,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr


def test_without_torch():
    run(WITHOUT)


def test_torch_is_imported_by_the_calls_that_take_tensors():
    run(LAZY)
