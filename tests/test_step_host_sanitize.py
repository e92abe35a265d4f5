"""The host code of include/exl3_step.h (checks, choice of kernels, splits,
workspaces) built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer and driven over many sizes
(tests/host_sanitize/step_driver.cpp), launchers and HIP calls replaced by
stand-ins that check what they are given; and the passes that calls with shared
prefixes make.  CPU only."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_sanitize")
CSRC = os.path.join(ROOT, "linear_exl3_input_amd", "csrc")
GXX = shutil.which("g++")
HIP_INC = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(GXX is None or not os.path.isdir(HIP_INC), reason="g++ or the HIP headers missing")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("step") / "step_sanitize")
    srcs = [os.path.join(CSRC, f) for f in ("exl3_host.cpp", "attn_host.cpp", "step_host.cpp")]
    srcs += [os.path.join(HERE, f) for f in ("stubs.cpp", "attn_stubs.cpp", "step_stubs.cpp", "step_driver.cpp")]
    cmd = [GXX, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC, "-I", os.path.join(ROOT, "include"), *srcs, "-o", exe, "-lpthread"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-4000:]

    def run(*args):
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([exe, *map(str, args)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env, timeout=600)
        assert "runtime error" not in r.stdout and "AddressSanitizer" not in r.stdout, r.stdout[-4000:]
        assert r.returncode == 0, r.stdout[-4000:]
        return r.stdout

    return run


def test_step_host_code_under_sanitizers(driver):
    assert "host checks done: 0 failures" in driver()


# batch, tokens, groups, query heads, key/value heads, head size, bits, columns of a page table of 16 tokens a page
@pytest.mark.parametrize("sizes,want", [
    ((4, 4, 1, 32, 8, 128, 16, 70), "plain none none whole"),        # few sequences: one plain launch
    ((64, 64, 1, 32, 8, 128, 8, 1600), "shared tile small whole"),
    ((64, 64, 64, 32, 8, 128, 8, 1600), "plain none none whole"),    # a group to each sequence
    ((8, 8, 1, 32, 8, 128, 8, 4000), "shared small small split"),
    ((3, 210, 1, 32, 8, 128, 16, 6000), "shared tile tile split"),
    ((16, 16, 1, 24, 4, 256, 4, 6000), "shared small small split"),
    ((16, 2048, 1, 32, 8, 128, 8, 6000), "shared tile tile split"),  # 512 rows of a sequence on each key/value head
    ((16, 2052, 1, 32, 8, 128, 8, 6000), "plain none none whole")])  # and 513
def test_the_passes_of_a_call_with_shared_prefixes(driver, sizes, want):
    assert driver(*sizes).split() == want.split()


@pytest.mark.parametrize("sizes,want", [
    ((2048, 32768, 8, 32, 8, 128, 8, 600), "shared tile small whole"),   # 0.6 GB of state
    ((16384, 16384, 16, 32, 8, 128, 8, 300), "shared tile small whole"),
    ((2048, 65536, 8, 32, 8, 128, 8, 600), "plain none none whole"),     # 1.1 GB
    ((2048, 131072, 1, 64, 8, 128, 8, 600), "plain none none whole"),    # 4.5
    ((16384, 1048576, 1, 64, 8, 128, 8, 600), "plain none none whole"),  # 35
    ((65536, 65536, 1, 64, 8, 128, 8, 300), "plain none none whole")])   # 2.3
def test_calls_whose_state_would_be_too_large_are_plain(driver, sizes, want):
    assert driver(*sizes).split() == want.split()


@pytest.mark.parametrize("bits,d,hkv,page", [(16, 64, 1, 16), (8, 128, 2, 64), (4, 256, 8, 256)])
def test_the_wide_tables_of_the_gpu_tests_make_a_call_share(driver, bits, d, hkv, page):
    """test_gpu_step_prefix.widened's number of columns, for two sequences and one group."""
    row = d * bits // 8 + (d // 32 if bits < 16 else 0)
    columns = int(200e6 / (page * hkv * 2 * row)) + 1
    assert driver(2, 2, 1, hkv, hkv, d, bits, columns * page // 16).split()[0] == "shared"
