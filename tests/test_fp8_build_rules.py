"""What the build refuses of the kernels over 8-bit floating-point operands.
CPU only: nothing is run."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mmvq_q2_gb300", "csrc")


def front_end(tmp_path, change):
    """What the compiler says to a changed copy of fp8_gemm.cu, without code for the device."""
    from mmvq_q2_gb300 import build
    root = tmp_path / "pkg" / "csrc"
    shutil.copytree(CSRC, root)
    shutil.copytree(os.path.join(os.path.dirname(os.path.dirname(CSRC)), "include"), tmp_path / "include")
    text = (root / "fp8_gemm.cu").read_text()
    changed = change(text)
    (root / "fp8_gemm.cu").write_text(changed)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "--cuda",
                        str(root / "fp8_gemm.cu"), "-o", str(tmp_path / "out.ii")], capture_output=True, text=True)
    return text != changed, r.returncode, r.stdout + r.stderr


def test_fp8_gemm_as_it_is(tmp_path):
    changed, rc, said = front_end(tmp_path, lambda s: s)
    assert not changed and rc == 0, said


@pytest.mark.parametrize("more", [2048, 8192])
def test_fp8_gemm_with_fewer_stages_than_accumulators(tmp_path, more):
    """One barrier tells that a stage is free and that an accumulator is full, which needs a stage for each accumulator.
    The 64-column form has less than 2 KB of shared memory to spare until it has one too few."""
    changed, rc, said = front_end(
        tmp_path, lambda s: s.replace("struct GemmShared {", "struct GemmShared {\n    char more[%d];" % more))
    assert changed and rc != 0 and "fewer stages than accumulators" in said, said
