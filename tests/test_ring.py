"""The page ring of the mma.sync decode kernel, replayed on the CPU (tests/ring_check.cu): for every shape's ring, no wait
passes before its page has landed, whatever warp or copy is late."""
import os
import subprocess

import pytest

from quantized_paged_kv_cache_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_check")
    subprocess.run([_build.nvcc(), "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    "-o", exe, os.path.join(HERE, "ring_check.cu")], check=True, capture_output=True)
    return lambda *a: subprocess.run([exe, *map(str, a)], capture_output=True, text=True, timeout=600).stdout.split()


def test_no_wait_passes_early_on_any_shape(check):
    out = check()
    assert out[-2:] == ["bad", "0"] and int(out[-3]) > 50, " ".join(out)


@pytest.mark.parametrize("stages,teams,bpp", [(23, 8, 1), (7, 8, 3), (5, 8, 4), (29, 8, 1), (11, 4, 2), (4, 8, 5)])
def test_the_replay_sees_a_ring_that_is_no_whole_number_of_rounds(check, stages, teams, bpp):
    assert check(stages, teams, bpp, 0) == ["bad"]
    assert check(stages, teams, bpp, 1) == ["good"]
