"""GPU: the attention kernel for many rows where smaller calls do not reach it:
heads of 256 over every cache format, caches past 4 GB, tiles whose keys are
split.  That each call runs on this kernel is checked in
test_attention_choice.py (attn_tile_cases.py has the sizes)."""
import math

import pytest
import torch

import attn_reference as ref
import attn_tile_cases as cases
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
FORMATS = [(b, t) for b in (16, 8, 4) for t in (BF16, F16)]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


class Call:
    """A call of attn_tile_cases over a cache whose unused slots are NaN, and its definition on a sample of rows."""

    def __init__(self, c, bits, dtype, page, holes=False, seed=0):
        g = torch.Generator().manual_seed(seed + c["d"] + bits)
        hq, hkv, d = c["hq"], c["hkv"], c["d"]
        self.c, self.dtype, self.page = c, dtype, page
        per = [-(-n // page) for n in c["kv_lens"]]
        pages = sum(per) + 2
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(per), max(per) + 1), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(per):
            self.table[i, :n] = order[at:at + n].int()
            at += n
        if holes:
            self.table[0, 3] = -1
            self.table[0, per[0] - 2] = pages + 5
        self.cache = ex.KvCache.empty(pages, page, hkv, d, bits, dtype)
        nan = torch.full((page, hkv, d), math.nan, dtype=dtype, device="cuda")
        for i in range(pages):
            ex.cache_write(self.cache, nan, nan, torch.arange(i * page, (i + 1) * page, dtype=torch.int32, device="cuda"))
        self.kv = []
        for i, n in enumerate(c["kv_lens"]):
            k, v = (torch.randn((n, hkv, d), generator=g).to(dtype) for _ in range(2))
            seq, pos = torch.full((n,), i, device="cuda"), torch.arange(n, device="cuda")
            ex.cache_write(self.cache, k.cuda(), v.cuda(), self.cache.slots(self.table.cuda(), seq, pos))
            self.kv.append((k, v))
        self.q = torch.randn((sum(c["q_lens"]), hq, d), generator=g).to(dtype)
        self.cu = torch.tensor([0] + c["q_lens"]).cumsum(0)

    def run(self, **kw):
        return ex.paged_attention(self.cache, self.q.cuda(), self.cu.int().cuda(), ints(self.c["kv_lens"]), self.table.cuda(), **kw)

    def check(self, got, window=0, rows=None):
        got = got.cpu()
        assert torch.isfinite(got).all()
        for i, (n, m) in enumerate(zip(self.c["q_lens"], self.c["kv_lens"])):
            at = torch.arange(n) if rows is None else torch.linspace(0, n - 1, min(n, rows)).long().unique()
            seen = ref.mask(n, m, True, window, self.table[i], self.page, self.cache.pages)[at]
            k, v = (ref.quantise(x, self.cache.bits) for x in self.kv[i])
            o, b = ref.attend(self.q[self.cu[i] + at].double(), k, v, seen, self.c["d"] ** -0.5, self.dtype)
            ref.check(got[self.cu[i] + at], o, b, f"sequence {i}")


@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_chunks_with_heads_of_256(bits, dtype):
    banner(f"chunks, heads of 256, {bits} bits {dtype}")
    x = Call(cases.CHUNKS, bits, dtype, 16)
    x.check(x.run())
    x.check(x.run(window=90), window=90)


@pytest.mark.parametrize("bits,dtype,d", [(16, BF16, 64), (4, F16, 64), (8, BF16, 128), (16, F16, 128), (4, BF16, 128),
                                          (8, F16, 256), (16, BF16, 256), (4, BF16, 256)])
def test_split_tiles_over_a_cache(bits, dtype, d):
    banner(f"split tiles, heads of {d}, {bits} bits {dtype}")
    x = Call(cases.LONG[d], bits, dtype, 64, holes=True)
    first = x.run()
    x.check(first, rows=12)
    x.check(x.run(window=6001), window=6001, rows=12)
    for _ in range(3):
        assert same_bits(x.run(), first)


@pytest.mark.parametrize("bits,dtype,d", [(8, BF16, 64), (16, BF16, 128), (4, F16, 128), (8, F16, 256)])
def test_more_tiles_than_the_gpu_holds(bits, dtype, d):
    banner(f"many tiles, heads of {d}, {bits} bits {dtype}")
    x = Call(cases.FULL[d], bits, dtype, 128)
    x.check(x.run(), rows=3)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F16, 64), (F16, 128), (BF16, 128), (BF16, 256), (F16, 256)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1500), (False, 0)])
def test_split_tiles_of_prompts(dtype, d, causal, window):
    banner(f"split prompts, heads of {d} {dtype} causal={causal} window={window}")
    c = cases.PROMPTS[d]
    g = torch.Generator().manual_seed(d)
    t = sum(c["q_lens"])
    q = torch.randn((t, c["hq"], d), generator=g).to(dtype)
    k, v = (torch.randn((t, c["hkv"], d), generator=g).to(dtype) for _ in range(2))
    cu = torch.tensor([0] + c["q_lens"]).cumsum(0)
    dev = (q.cuda(), k.cuda(), v.cuda(), cu.int().cuda())
    got = ex.prompt_attention(*dev, causal=causal, window=window)
    for i, n in enumerate(c["q_lens"]):
        at = torch.linspace(0, n - 1, 12).long()
        rows = slice(int(cu[i]), int(cu[i + 1]))
        o, b = ref.attend(q[cu[i] + at].double(), k[rows].double(), v[rows].double(), ref.mask(n, n, causal, window)[at], d ** -0.5,
                          dtype)
        ref.check(got.cpu()[cu[i] + at], o, b, f"sequence {i}")
    for _ in range(3):
        assert same_bits(ex.prompt_attention(*dev, causal=causal, window=window), got)


def test_tiles_over_a_cache_past_four_gigabytes():
    c = cases.FAR
    pages, page, heads, d, (n,), (m,) = 5200, 256, c["hkv"], c["d"], c["q_lens"], c["kv_lens"]
    banner(f"far pages, {n} rows")
    cache = ex.KvCache.empty(pages, page, heads, d, 16, BF16)
    assert cache.k.numel() * 2 > 2 ** 32
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn((x, heads, d), generator=g).to(BF16) for x in (m, m, n))
    table = ints([[pages - 1, 4100]])
    slots = cache.slots(table, torch.zeros(m, dtype=torch.int32, device="cuda"), torch.arange(m, dtype=torch.int32, device="cuda"))
    ex.cache_write(cache, k.cuda(), v.cuda(), slots)
    got = ex.paged_attention(cache, q.cuda(), ints([0, n]), ints([m]), table)
    ref.check(got, *ref.attend(q.double(), k.double(), v.double(), ref.mask(n, m), d ** -0.5, BF16), "far pages")
