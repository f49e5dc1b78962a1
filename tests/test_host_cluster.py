"""How page selection is launched, against a fake CUDA runtime (tests/cluster_check.cu), on the CPU."""
import os
import subprocess

import pytest

from quantized_paged_kv_cache_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cluster") / "cluster_check")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    "-o", exe, os.path.join(HERE, "cluster_check.cu")], check=True, capture_output=True)
    return lambda n: [line.split() for line in subprocess.run([exe, str(n)], capture_output=True, text=True, timeout=600).stdout.splitlines()]


def test_where_sixteen_blocks_fit(check):
    out = check(9)
    assert [x[:2] for x in out] == [["1", "16"]] * 4 + [["1", "4"], ["1", "16"]]
    assert all(int(x[2]) <= 200 * 1024 and x[3:] == ["0"] for x in out)


def test_where_they_do_not(check):
    out = check(0)
    assert len(out) == 6 and not any("bad" in x for x in out), out
    for launches, cluster, smem, ws in out:  # eight blocks at most, or two launches through the workspace
        assert (launches == "1" and int(cluster) <= 8 and int(smem) <= 200 * 1024 and ws == "0") or (launches == "2" and int(ws) > 0)
    assert [x[1] for x in out[:3]] == ["8", "8", "8"]
