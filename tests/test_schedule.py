"""The GEMMs' division of tiles and K slabs among CTAs (csrc/schedule.cuh), checked
on the host: the schedule that the W8A16 kernel walks against the list of split tiles
that its fix-up is given. Compiled with nvcc as host code (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

import test_feed_forward
import test_split_forms as split_forms

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    """Runs tests/native/schedule_check.cu with the given arguments."""
    exe = tmp_path_factory.mktemp("schedule") / "schedule_check"
    csrc = os.path.join(ROOT, "block_scaled_fp8_fp8blk_b200", "csrc")
    subprocess.run([NVCC, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-I", csrc, "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    os.path.join(HERE, "native", "schedule_check.cu")], check=True)

    def run(*args):
        out = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=300)
        assert out.returncode == 0, out.stdout
        return out.stdout

    return run


pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def test_schedule_covers_every_slab_and_matches_the_split_tiles(check):
    assert check().startswith("ok")


@pytest.mark.parametrize("M,K,N", split_forms.W8A16_SPLIT + split_forms.W8A16_LAST_WAVE)
def test_the_w8a16_sizes_are_split(check, M, K, N):
    """The sizes of test_split_forms.py split tiles, with both epilogues."""
    for epilogue, n in ((1, N), (2, N // 2)):
        assert int(check("w8a16", epilogue, M, n, K).split()[1]) > 0


def test_both_sides_of_the_whole_tile_rule(check):
    """Whole tiles where the split would save less than its fix-up."""
    assert check("w8a16", 1, 48, 1000, 640).split() == ["8", "0"]
    assert check("w8a16", 0, 48, 1000, 640).split() != ["8", "0"]       # the plain linear always splits


# Clusters of 2, 4 and 8 CTAs that a B200 may hold at once (of 74, 37 and 18 at most:
# a cluster lies within one group of SMs, and the groups' sizes differ from GPU to GPU).
RESIDENT = [(74, r4, r8) for r4 in (30, 33, 35, 37) for r8 in (12, 15, 18)]


@pytest.mark.parametrize("resident", RESIDENT)
@pytest.mark.parametrize("epilogue", [1, 2])
def test_the_w8a8_sizes_reach_every_cluster_size(check, epilogue, resident):
    def split(M, K, N):
        return int(check("w8a8", epilogue, M, N if epilogue == 1 else N // 2, K, *resident))

    assert all(split(*size) == 2 for size in split_forms.W8A8_TWO)
    sizes = test_feed_forward.SPLIT_SHAPES + test_feed_forward.LINEAR_SHAPES + split_forms.W8A8_TWO
    assert {split(*size) for size in sizes} == {1, 2, 4, 8}
