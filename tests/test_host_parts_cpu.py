"""Host-only parts of the library compiled against a stand-in for the CUDA
runtime (tests/host/cuda_runtime.h) and run: no GPU, no toolkit."""
import os
import shutil
import subprocess

import pytest

import mixed_precision_dense_sm_gb300 as lib

HOST = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")
CXX = shutil.which("g++") or shutil.which("c++")


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
@pytest.mark.parametrize("name", sorted(f[:-4] for f in os.listdir(HOST) if f.endswith(".cpp")))
def test_host_part(name, tmp_path):
    exe = str(tmp_path / name)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", HOST, "-I",
                    os.path.join(lib.HERE, "csrc"), os.path.join(HOST, name + ".cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
