"""GPU: caches of codes that the caller filled, with what cache_write never
stores: e4m3's NaN codes and scales whose values overflow the 16-bit type.
They must reach the rows that see them and no others, in both kernels."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
# (type, bits): a scale byte at which the largest code, 448 or 6, is past the type's range
OVER = {(BF16, 8): 250, (BF16, 4): 254, (F16, 8): 136, (F16, 4): 142}


def values(code, scale, dtype):
    """What the format says codes [.., d * bits / 8] and scales [.., d / 32] are, rounded to the type, in float64."""
    if code.shape[-1] == 32 * scale.shape[-1]:
        v = code.view(torch.float8_e4m3fn).double()
    else:
        grid = torch.tensor(ref.E2M1 + tuple(-x for x in ref.E2M1), dtype=torch.float64)
        v = grid[torch.stack((code & 15, code >> 4), -1).flatten(-2).long()]
    v = v.unflatten(-1, (-1, 32)) * torch.exp2(scale.double() - 127)[..., None]
    return v.flatten(-2).to(dtype).double()


def codes(g, shape, d, dtype, bits):
    """Random finite codes, and scales that give values of about one."""
    code = torch.randint(0, 256, (*shape, d * bits // 8), generator=g, dtype=torch.uint8)
    if bits == 8:
        code = (code & 0x80) | 0x28 | (code & 0x17)  # 0.25 .. 3.75
    return code, torch.randint(125, 128, (*shape, d // 32), generator=g, dtype=torch.uint8)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [6, 90])  # 6 rows of a group of 2 on the kernel for few rows, 90 on the tiles of 128
def test_codes_that_are_not_finite_stay_with_the_rows_that_see_them(n, d, bits, dtype):
    banner(f"foreign codes n={n} d={d} {bits} bits {dtype}")
    hq, hkv, page, lens = 4, 2, 32, [150, 300]
    g = torch.Generator().manual_seed(n + d + bits)
    pages = sum(-(-m // page) for m in lens) + 1
    kc, ks = codes(g, (pages, hkv, page), d, dtype, bits)
    vc, vs = codes(g, (pages, hkv, page), d, dtype, bits)
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((2, 10), -1, dtype=torch.int32)
    table[0, :5], table[1, :10] = order[:5], order[5:15]
    q = torch.randn((2 * n, hq, d), generator=g).to(dtype)

    def at(seq, key):
        return int(table[seq, key // page]), key % page

    def overflow(code, scale, seq, key, head, block, value, sign):
        """One value past the range, the rest of its block zero."""
        pg, o = at(seq, key)
        scale[pg, head, o, block] = OVER[(dtype, bits)]
        code[pg, head, o, block * 4 * bits:(block + 1) * 4 * bits] = 0
        if bits == 8:
            code[pg, head, o, 32 * block + value] = 0x7E | sign << 7
        else:
            code[pg, head, o, 16 * block + value // 2] = (7 | sign << 3) << (4 * (value % 2))

    for s, m in enumerate(lens):
        overflow(vc, vs, s, m - n // 2 - 1, 0, 0, 5, 0)      # +inf, seen by the later half
        overflow(vc, vs, s, m - n // 3 - 1, 0, 1, 30, 1)     # -inf
        overflow(vc, vs, s, m - 1, 1, d // 32 - 1, 31, 1)    # the last row's own
        overflow(kc, ks, s, m - n // 4 - 1, 1, 0, 3, 0)
        pg, o = at(s, m - 2)
        vs[pg, 1, o, 0] = 255
        if bits == 8:
            pg, o = at(s, m - n // 2 - 1)
            vc[pg, 1, o, 9], vc[pg, 1, o, d - 1] = 0x7F, 0xFF
            pg, o = at(s, m - n // 5 - 1)
            kc[pg, 0, o, d - 2] = 0x7F
    cache = ex.KvCache(*(t.cuda() for t in (kc, vc, ks, vs)), dtype)
    k, v = values(kc, ks, dtype), values(vc, vs, dtype)
    v[..., :32][vs[..., 0] == 255] = math.nan
    got = ex.paged_attention(cache, q.cuda(), torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    for s, m in enumerate(lens):
        key = torch.arange(m)
        pg, o = table[s, key // page].long(), key % page
        want, bound = ref.attend(q[s * n:(s + 1) * n].double(), k[pg, :, o], v[pg, :, o], ref.mask(n, m), d ** -0.5, dtype)
        assert torch.isfinite(want[0]).all() and not torch.isfinite(want[-1]).all()
        ref.check(got[s * n:(s + 1) * n], want, bound, f"sequence {s}")


@pytest.mark.parametrize("bits,dtype", [(8, BF16), (8, F16), (4, BF16), (4, F16)])
def test_every_scale_byte_reads_back_as_the_power_it_names(bits, dtype):
    """0 and 1 (below fp32's normal range) and those past the type's range among them."""
    code = (torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 256) if bits == 8 else
            torch.arange(128, dtype=torch.uint8).view(1, 1, 1, 128)).expand(16, 1, 16, -1).contiguous()
    scale = torch.arange(256).to(torch.uint8).view(16, 1, 16, 1).expand(16, 1, 16, 8).contiguous()
    cache = ex.KvCache(code.cuda(), code.cuda(), scale.cuda(), scale.cuda(), dtype)
    k, v = ex.cache_read(cache, torch.arange(256, dtype=torch.int32, device="cuda"))
    want = values(code, scale, dtype).reshape(256, 1, 256)
    want[255] = math.nan
    for got in (k, v):
        assert torch.equal(got.cpu().double().nan_to_num(1e300, 2e300, -2e300), want.nan_to_num(1e300, 2e300, -2e300))
