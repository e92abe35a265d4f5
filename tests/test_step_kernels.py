"""The attention kernels that the built library holds are those that calls reach
(host only, no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

import linear_exl3_input_amd as ex

pytestmark = pytest.mark.skipif(not os.path.exists(ex.lib_path()) or shutil.which("nm") is None, reason="libexl3.so not built, or no nm")

PLAIN, SINKS, SHARED, OWN = range(4)


def held(kernel):
    """(heads, bits, the kernel's other numbers) of every instance."""
    text = subprocess.run(["nm", "-C", ex.lib_path()], stdout=subprocess.PIPE, text=True, check=True).stdout
    found = re.findall(rf" exl3::{kernel}<(true|false), ([^>]*)>\(", text)
    return sorted({(t == "true", *(int(n) for n in re.findall(r"\b(?:\(exl3::AttnKind\))?(\d+)\b", rest))) for t, rest in found})


def wanted(columns):
    """Packed rows (0 bits) have no shared prefixes; two columns of 16 rows are for narrow heads, and not for own keys."""
    out = []
    for bf16 in (True, False):
        for d in (64, 128, 256):
            for kind in (PLAIN, SINKS, SHARED, OWN):
                for bits in (16, 8, 4) if kind in (SHARED, OWN) else (0, 16, 8, 4):
                    if columns is None:
                        out.append((bf16, d, bits, kind))
                    else:
                        out += [(bf16, d, bits, n, kind) for n in (1, 2) if n == 1 or (d < 256 and kind != OWN)]
    return sorted(out)


def test_small_kernels():
    assert held("attn_small_kernel") == wanted(2)


def test_tile_kernels():
    assert held("attn_tile_kernel") == wanted(None)
