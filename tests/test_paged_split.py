"""The paged attention kernels' split of key work over their blocks, on the
host: tests/line_split.cpp runs the kernels' own source (paged_line.cuh) on an
emulated warp and checks that every unit of keys is taken exactly once."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("split") / "line_split")
    subprocess.run(
        ["g++", "-std=c++17", "-O2", "-Wall", "-Wno-unknown-pragmas",
         "-I", os.path.join(ROOT, "prefill_blockwise_int8_b200", "csrc"),
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(CUDA, "include"),
         os.path.join(ROOT, "tests", "line_split.cpp"), "-o", exe], check=True)

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stdout
    return run


@pytest.mark.parametrize("new,lens", [
    ("1,0", "4096,2000"),          # an idle sequence last
    ("0,1", "2000,4096"),          # and first
    ("1,0", "1000,2000"),          # idle keys outnumber the active ones
    ("0,1,0", "9000,50,9000"),
    ("0,0,0", "1000,2000,3"),      # nobody active
    ("0,5,0,0,700,0", "40,5,6000,0,900,1"),
    ("0," * 33 + "1," + "0," * 33 + "2", "900," * 33 + "7," + "900," * 33 + "800"),
    ("1,1", "0,1"),
    ("9,300", "3,200"),            # fewer keys than new tokens
])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("hkv,group", [(8, 4), (1, 1), (2, 24)])
def test_every_unit_is_taken_once(split, new, lens, hkv, group, causal):
    most = max(map(int, new.split(",")))
    split("-", new, lens, hkv, group, causal, most)


@pytest.mark.parametrize("seed", [1, 2])
def test_random_batches(split, seed):
    split(seed, 25)
