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


def test_launchers_remember_nothing_per_process():
    """A function-local static of a launcher is a lock, a table of devices or a
    limit per device: the attributes it stands for belong to a device."""
    import re
    csrc = os.path.join(lib.HERE, "csrc")
    bad = []
    for f in sorted(os.listdir(csrc)):
        if not f.endswith((".cu", ".cuh", ".h")):
            continue
        for line in open(os.path.join(csrc, f)):
            m = re.match(r"\s+static (?!constexpr|const |_?_?inline)([\w:<>\[\], ]+?)\s+\w+(\[[^\]]*\])*( = .*)?;", line)
            if m and not re.match(r"(std::mutex|DeviceLimits|(gemm103::)?(DeviceLimits|PerDevice<.*>))$", m.group(1)):
                if "kMaxDevices]" not in line:
                    bad.append((f, line.strip()))
    assert not bad, bad


def test_operand_descriptors_start_from_zero():
    """A field of an operand's description that a plan does not set reads as zero
    (the paired copy takes the source's columns from one)."""
    import re
    text = open(os.path.join(lib.HERE, "csrc", "api.cu")).read()
    local = re.findall(r"^ +OperandDesc (\w[^;(&*]*);", text, flags=re.M)
    local = [d for decl in local for d in re.split(r",\s*", decl) if decl != "a, b"]
    assert local and all(d.endswith("{}") for d in local), local
