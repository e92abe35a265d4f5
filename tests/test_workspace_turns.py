"""Host threads whose calls share a workspace (as the binding's calls on one
stream do): a call's launches follow one another
(tests/host_sanitize/turns.cpp).  CPU only."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_exl3_input_amd", "csrc")
GXX = shutil.which("g++")
HIP_INC = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(GXX is None or not os.path.isdir(HIP_INC), reason="g++ or the HIP headers missing")


def test_no_launches_between_those_of_a_call(tmp_path):
    exe = str(tmp_path / "turns")
    srcs = [os.path.join(CSRC, f) for f in ("exl3_host.cpp", "attn_host.cpp", "step_host.cpp")]
    cmd = [GXX, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           "-I", HIP_INC, "-I", os.path.join(ROOT, "include"), *srcs, os.path.join(ROOT, "tests", "host_sanitize", "turns.cpp"),
           "-o", exe, "-lpthread"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-4000:]
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0 and "runtime error" not in r.stdout and "AddressSanitizer" not in r.stdout, r.stdout[-4000:]
