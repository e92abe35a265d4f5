"""Bounds of the packed prompts' loads in the built kernels (host only, no GPU).

The tile kernel reads packed keys and values through a buffer descriptor that
ends with a tile's last key, and relies on it: rows past the end of a sequence,
which can be past the end of the caller's tensors, must read as zeros.  The
scalar offset of a buffer instruction takes no part in that check (or makes the
descriptor's size wrap below zero), so a row's place has to be in the vector
offset.  This test compiles the kernels to gfx950 assembly and looks at every
buffer access."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from linear_exl3_input_amd import build as b

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")

# op, data, vector offset, descriptor, scalar offset
ACCESS = re.compile(r"^\s*(buffer_(?:load|store)_\w+)\s+[av]\S*,\s*(\S+),\s*(s\[\d+:\d+\]),\s*(\S+)(.*)$", re.M)


def accesses(asm):
    """(instruction, scalar offset, whether the vector offset is used) of every buffer access through a descriptor of
    the kernel's own; register spills go through the scratch descriptor without an offset register."""
    return [(m.group(0).strip(), m.group(4), "offen" in m.group(5)) for m in ACCESS.finditer(asm)]


def _asm(d, tmp):
    src, out = os.path.join(tmp, f"tile_{d}.hip"), os.path.join(tmp, f"tile_{d}.s")
    with open(src, "w") as f:
        f.write('#include "attn_tile.hpp"\n'
                f"template __global__ void exl3::attn_tile_kernel<true, {d}, 0>(exl3::AttnParams);\n")
    flags = [f for f in (*b.COMMON, *b.EXTRA[f"attn_d{d}.hip"]) if f != "-fPIC"]
    subprocess.run([HIPCC, *flags, "-I", b.CSRC, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    return open(out).read()


def test_packed_loads_have_their_row_in_the_checked_offset(tmp_path):
    with ThreadPoolExecutor(3) as ex:
        for d, asm in zip((64, 128, 256), ex.map(lambda d: _asm(d, str(tmp_path)), (64, 128, 256))):
            found = [x for x in accesses(asm) if "offen" in x[0]]
            assert len(found) >= 24, f"heads of {d}: {len(found)} buffer accesses"  # a tile's 4 + 8 loads, twice
            bad = [text for text, scalar, _ in found if scalar != "0"]
            assert not bad, f"heads of {d}: {len(bad)} of {len(found)} with a scalar offset, e.g. {bad[:2]}"


def test_the_look_at_accesses_sees_a_scalar_offset():
    asm = ("\tbuffer_load_dwordx4 v[2:5], v1, s[8:11], 0 offen\n\tbuffer_load_dwordx2 v[6:7], v1, s[8:11], s3 offen\n"
           "\tbuffer_store_dword v9, off, s[0:3], 0 offset:4\n")
    assert [(s, o) for _, s, o in accesses(asm)] == [("0", True), ("s3", True), ("0", False)]
