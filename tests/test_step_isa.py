"""Bounds of the packed prompts' loads in the built kernels with first tokens
beside a window (host only, no GPU): as in test_attention_isa, a row's place is
in the offset that the buffer descriptor checks."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

from linear_exl3_input_amd import build as b
from test_attention_isa import HIPCC, accesses, pytestmark  # noqa: F401


def _asm(d, tmp):
    src, out = os.path.join(tmp, f"sinks_{d}.hip"), os.path.join(tmp, f"sinks_{d}.s")
    with open(src, "w") as f:
        f.write('#include "attn_tile.hpp"\n'
                f"template __global__ void exl3::attn_tile_kernel<true, {d}, 0, exl3::ATTN_SINKS>(exl3::AttnParams);\n")
    flags = [f for f in (*b.COMMON, *b.EXTRA[f"attn_sinks_d{d}.hip"]) if f != "-fPIC"]
    subprocess.run([HIPCC, *flags, "-I", b.CSRC, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    return open(out).read()


def test_packed_loads_have_their_row_in_the_checked_offset(tmp_path):
    with ThreadPoolExecutor(3) as ex:
        for d, asm in zip((64, 128, 256), ex.map(lambda d: _asm(d, str(tmp_path)), (64, 128, 256))):
            found = [x for x in accesses(asm) if "offen" in x[0]]
            assert len(found) >= 24, f"heads of {d}: {len(found)} buffer accesses"
            bad = [text for text, scalar, _ in found if scalar != "0"]
            assert not bad, f"heads of {d}: {len(bad)} of {len(found)} with a scalar offset, e.g. {bad[:2]}"
