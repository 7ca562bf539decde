"""Which positions a row of the attention operators sees, checked on the CPU:
the kernels' functions, compiled for the host with checks of signed overflow
(tests/kv_probe.cu), against 64-bit arithmetic at the ends of their ranges
(padding rows far before the first position, no window, the longest cache)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_positions_that_rows_see(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "kv_probe")
    subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler", "-fno-sanitize-recover=all",
                    f"-I{os.path.join(ROOT, 'skinny_bf16_gemm_residual_gb300', 'csrc')}", f"-I{os.path.join(ROOT, 'include')}",
                    os.path.join(ROOT, "tests", "kv_probe.cu"), "-o", exe, "-lubsan"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) > 500
