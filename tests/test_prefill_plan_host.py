"""The prompt attention's division of work, on the CPU: the very functions of the plan kernel, the blocks'
walk and the join (prefill.cuh), compiled for the host with the shipped tiles and costs, against brute
force (prefill_plan_host.cu): every kv tile of every unit is read once, every cut unit is named once with
all the blocks that hold its pieces, shares are equal within the moves of their ends, and the closed-form
sums agree in 32 and 64 bits."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from paged_kv_decode_np_gb300 import build_lib
    out = str(tmp_path_factory.mktemp("plan") / "prefill_plan_host")
    cmd = [build_lib.nvcc(), "-std=c++17", "-O2", *build_lib.ARCH, "-I", build_lib.INCLUDE, "-I", build_lib.CSRC,
           os.path.join(ROOT, "tests", "prefill_plan_host.cu"), "-o", out]
    p = subprocess.run(cmd, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    return out


@pytest.mark.parametrize("seed", range(4))
def test_shares_cover_every_tile_once(program, seed):
    p = subprocess.run([program, str(seed), "300"], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stdout == "ok\n", p.stdout
