"""The kernel that the GPU tests' calls run on (tests/attn_tile_cases.py): the
host's choice, asked of its code built with g++ and stand-ins for the launches
(tests/host_sanitize/attn_which.cpp).  CPU only."""
import os
import shutil
import subprocess

import pytest

import attn_tile_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_sanitize")
CSRC = os.path.join(ROOT, "linear_exl3_input_amd", "csrc")
GXX = shutil.which("g++")
HIP_INC = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(GXX is None or not os.path.isdir(HIP_INC), reason="g++ or the HIP headers missing")


@pytest.fixture(scope="module")
def which(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("attn") / "which")
    srcs = [os.path.join(CSRC, "exl3_host.cpp"), os.path.join(CSRC, "attn_host.cpp"), os.path.join(HERE, "stubs.cpp"),
            os.path.join(HERE, "attn_stubs.cpp"), os.path.join(HERE, "attn_which.cpp")]
    subprocess.run([GXX, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC, "-I", os.path.join(ROOT, "include"), *srcs,
                    "-o", exe, "-lpthread"], check=True)

    def ask(c):
        args = [int(c["prompt"]), len(c["q_lens"]), sum(c["q_lens"]), c["hq"], c["hkv"], c["d"]]
        r = subprocess.run([exe, *map(str, args)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout.split()

    return ask


@pytest.mark.parametrize("case", cases.ALL, ids=lambda c: c["name"])
def test_the_call_runs_on_the_tile_kernel(which, case):
    assert which(case) == ["tile", "split" if case["split"] else "whole"]


def test_few_rows_run_on_the_small_kernel(which):
    for d in (64, 128, 256):
        assert which(cases.call("one token", [1], [9000], 32, 8, d, True)) == ["small", "split"]
