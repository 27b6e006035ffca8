"""The products' bounded waits (csrc/mbar_wait.cuh), compiled for the host: a
wait that runs out while the phase completes for some of the lanes must end in
the same way for every lane of a warp, and for every warp of a group, as barriers
and warp-wide instructions follow it."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp4_post_weight_grid_b200", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("waits") / "waits")
    subprocess.run([cxx, "-O1", "-std=c++20", "-pthread", "-I", CSRC, os.path.join(HERE, "native", "mbar_wait_host.cpp"),
                    "-o", out], check=True, timeout=300)
    return out


@pytest.mark.parametrize("scenario,warps,group,dead", [
    (0, [32] * 4, 128, 0),              # complete
    (1, [0] * 4, 0, 1),                 # never complete
    (2, [0] * 4, 0, 1),                 # seen by half of each warp's lanes when time runs out
    (3, [32, 32, 0, 32], 0, 1),         # seen by three of the four warps
    (4, [32] * 4, 128, 0),              # complete after a while, a look earlier or later
])
def test_lanes_and_groups_agree(program, scenario, warps, group, dead):
    r = subprocess.run([program, str(scenario)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    want = "warps " + " ".join(map(str, warps)) + f" group {group} dead {dead}"
    assert r.stdout.strip() == want


def test_every_wait_of_the_kernels_is_one_of_these():
    for name in ("linear.cu", "matmul.cu", "product_tile.cuh", "few.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert not re.search(r"\bmbar_try\s*\(|try_wait|test_wait", text), name
