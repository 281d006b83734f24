"""How the chunk kernels' softmax warps leave when a wait gives up (CPU): the order of their waits and barriers,
from the kernel's own header, over simulated warps that give up at random moments, one by one."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SCHEDULES = 3000


@pytest.fixture(scope="module")
def simulate(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("soft") / "chunk_soft_host")
    subprocess.check_call([cxx, "-O1", "-std=c++17", "-o", exe, os.path.join(HERE, "chunk_soft_host.cpp")])

    def run(leave):
        out = subprocess.run([exe, str(SCHEDULES), str(leave)], capture_output=True, text=True, check=True).stdout
        return dict(zip(("hung", "gave_up", "split", "whole"), map(int, out.split())))

    return run


def test_all_warps_leave_together(simulate):
    r = simulate(0)
    assert r["hung"] == 0
    assert r["gave_up"] + r["whole"] == SCHEDULES and r["whole"] > SCHEDULES // 5
    assert r["split"] > SCHEDULES // 20  # one warp of a row gave up where the other went on


def test_the_simulation_sees_a_warp_that_leaves_its_partner(simulate):
    assert simulate(1)["hung"] > 0
