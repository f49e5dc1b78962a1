"""The kernels' shared-memory limits against a fake CUDA runtime (tests/limits_check.cu), on the CPU."""
import os
import subprocess

from quantized_paged_kv_cache_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_limits_are_never_taken_back(tmp_path):
    exe = str(tmp_path / "limits_check")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    "-o", exe, os.path.join(HERE, "limits_check.cu"), "-lpthread"], check=True, capture_output=True)
    assert subprocess.run([exe], capture_output=True, text=True, timeout=600).stdout.splitlines() == ["good"]
