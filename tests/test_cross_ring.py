"""The rings of the cross attention's read on the tensor cores, on the CPU: ``tests/cross_ring_check.cpp`` runs a model of
the kernel's waits with the kernel's own ring sizes (``csrc/cross_ring.h``) under random schedules."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_level_head_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("ring") / "cross_ring_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, os.path.join(ROOT, "tests", "cross_ring_check.cpp"), "-o", exe], check=True)

    def run(d, tiles, runs, buffers=0, sums=0):
        res = subprocess.run([exe, str(d), str(d // 32), str(buffers), str(sums), str(tiles), str(runs)], capture_output=True, text=True)
        assert res.returncode == 0
        return tuple(map(int, res.stdout.split()))   # buffers, sums, wrong runs, stuck runs

    return run


@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 9, 17])
@pytest.mark.parametrize("d", [64, 128])
def test_no_schedule_meets_another_tiles_values(model, d, tiles):
    buffers, sums, wrong, stuck = model(d, tiles, 1000)
    assert wrong == 0 and stuck == 0, f"{buffers} buffers, {sums} places of sums: {wrong} wrong, {stuck} stuck of 1000"


def test_the_model_sees_a_place_that_is_taken_too_early(model):
    """Fewer places than buffers: a warp a tile behind finds another tile's sum in one of them."""
    for buffers, sums in ((4, 3), (3, 2), (4, 2)):
        assert model(128, 9, 1000, buffers, sums)[2] > 0
    assert model(128, 9, 1000, 4, 4)[2:] == (0, 0)
