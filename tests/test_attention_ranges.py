"""The keys that the attention kernels' steps and page look-ups reach for any
length in device memory (tests/host_sanitize/attn_ranges.cpp), built with g++
under AddressSanitizer and UndefinedBehaviorSanitizer.  CPU only."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GXX = shutil.which("g++")
HIP_INC = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(GXX is None or not os.path.isdir(HIP_INC), reason="g++ or the HIP headers missing")


def test_no_key_leaves_32_bits(tmp_path):
    exe = str(tmp_path / "attn_ranges")
    cmd = [GXX, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           "-I", HIP_INC, os.path.join(ROOT, "tests", "host_sanitize", "attn_ranges.cpp"), "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-4000:]
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0 and " 0 bad" in r.stdout, r.stdout[-4000:]
