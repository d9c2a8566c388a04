"""The GEMMs' division of tiles and K slabs among CTAs (csrc/schedule.cuh), checked
on the host: the schedule that the W8A16 kernel walks against the list of split tiles
that its fix-up is given. Compiled with nvcc as host code (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

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
