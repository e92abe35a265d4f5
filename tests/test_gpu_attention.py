"""GPU: attention over the paged cache and over packed prompts, against the
definition in 64 bits (attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


class Paged:
    """A cache with every page that no sequence uses, and every slot past a sequence's end, full of NaN."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, dtype, bits, page, seed=0, gain=1.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.page, self.dtype = q_lens, kv_lens, page, dtype
        per = [-(-n // page) for n in kv_lens]
        pages = sum(per) + spare
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.full((len(kv_lens), max(per + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(per):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.cache = ex.KvCache.empty(pages, page, hkv, d, bits, dtype)
        nan = torch.full((pages * page, hkv, d), math.nan, dtype=dtype, device="cuda")
        ex.cache_write(self.cache, nan, nan, torch.arange(pages * page, dtype=torch.int32, device="cuda"))
        self.k = [normal(g, (n, hkv, d), dtype, gain) for n in kv_lens]
        self.v = [normal(g, (n, hkv, d), dtype) for n in kv_lens]
        self.q = normal(g, (sum(q_lens), hq, d), dtype)
        self.cu = torch.tensor([0] + q_lens).cumsum(0).int()
        self.write()

    def write(self):
        for i, n in enumerate(self.kv_lens):
            if n:
                p = torch.arange(n)
                slots = self.table[i, p // self.page].long() * self.page + p % self.page
                ex.cache_write(self.cache, self.k[i].cuda(), self.v[i].cuda(), slots.int().cuda())

    def run(self, **kw):
        return ex.paged_attention(self.cache, kw.pop("q", self.q.cuda()), self.cu.cuda(),
                                  torch.tensor(self.kv_lens, dtype=torch.int32).cuda(), self.table.cuda(), **kw)

    def expect(self, window=0, scale=None):
        bits = self.cache.bits
        d = self.q.shape[-1]
        out, bound = [], []
        for i, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            seen = ref.mask(n, m, True, window, self.table[i], self.page, self.cache.pages)
            o, b = ref.attend(self.q[self.cu[i]:self.cu[i + 1]].double(), ref.quantise(self.k[i], bits),
                              ref.quantise(self.v[i], bits), seen, d ** -0.5 if scale is None else scale, self.dtype)
            out.append(o)
            bound.append(b)
        return torch.cat(out), torch.cat(bound)


FORMATS = [(b, t, d) for b in (16, 8, 4) for t in (BF16, F16) for d in (64, 128, 256)]


@pytest.mark.parametrize("bits,dtype,d", FORMATS)
def test_paged_one_token(bits, dtype, d):
    """One new token a sequence: lengths 1 to several steps and pages, odd ones among them."""
    banner(f"paged one token {bits} {dtype} {d}")
    x = Paged([1] * 9, [1, 2, 31, 32, 33, 100, 129, 517, 1030], 8, 2, d, dtype, bits, 32, seed=d + bits)
    ref.check(x.run(), *x.expect(), f"{bits} bits")


@pytest.mark.parametrize("bits,dtype,d", FORMATS)
def test_paged_chunks(bits, dtype, d):
    """Chunks of new tokens, none at all for one sequence, longer than the tiles."""
    banner(f"paged chunks {bits} {dtype} {d}")
    x = Paged([5, 0, 17, 1, 64, 150], [70, 40, 17, 300, 65, 333], 6, 2, d, dtype, bits, 16, seed=d + bits + 1)
    ref.check(x.run(), *x.expect(), f"{bits} bits")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 7), (5, 1), (12, 1), (16, 1), (24, 2), (40, 1), (96, 8)])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_paged_groups(hq, hkv, n):
    banner(f"paged groups {hq}/{hkv} n={n}")
    x = Paged([n, 1, n], [n, 200, 3 * n + 130], hq, hkv, 64, BF16, 8, 64, seed=hq + n)
    ref.check(x.run(), *x.expect(), f"{hq}/{hkv}")


@pytest.mark.parametrize("window", [1, 5, 32, 100, 1000])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [9, 2, 40], [200, 1, 130]])
def test_paged_window(window, q_lens):
    banner(f"paged window {window} {q_lens}")
    x = Paged(q_lens, [210, 77, 640], 4, 2, 128, F16, 16, 16, seed=window)
    ref.check(x.run(window=window), *x.expect(window=window), f"window {window}")


@pytest.mark.parametrize("bits,d", [(16, 64), (8, 128), (4, 256), (16, 128)])
@pytest.mark.parametrize("n", [1, 30, 140])
def test_paged_holes_and_empty_rows(bits, d, n):
    """Pages that are missing, a whole sequence without any, rows before the sequence's start, no keys at all."""
    banner(f"paged holes {bits} {d} n={n}")
    x = Paged([n, n, n, 1], [300, 200, max(0, n - 10), 0], 4, 1, d, BF16, bits, 16, seed=n)
    x.table[0, 2] = -1
    x.table[0, 7] = x.cache.pages  # out of range
    x.table[0, 11:14] = -7
    x.table[1] = -1
    got = x.run()
    want, bound = x.expect()
    ref.check(got, want, bound, "holes")
    assert not got[n:2 * n].any()  # no pages
    assert not got[3 * n:].any()  # no keys
    if n > 10:
        assert not got[2 * n:2 * n + 10].any()  # before the first key


def test_paged_table_narrower_than_the_lengths():
    x = Paged([1, 1], [100, 60], 4, 2, 64, BF16, 16, 16, seed=3)
    x.table = x.table[:, :4].contiguous()
    ref.check(x.run(), *x.expect(), "narrow table")
    wide = torch.full((2, 40), -1, dtype=torch.int32)
    wide[:, 5:9] = x.table
    x.table = wide.cuda()[:, 5:9].cpu()
    got = ex.paged_attention(x.cache, x.q.cuda(), x.cu.cuda(), torch.tensor(x.kv_lens, dtype=torch.int32).cuda(),
                             wide.cuda()[:, 5:9])
    ref.check(got, *x.expect(), "strided table")


@pytest.mark.parametrize("bits,dtype,d", [(16, BF16, 128), (16, F16, 64), (8, BF16, 64), (16, BF16, 256), (4, F16, 128)])
@pytest.mark.parametrize("n", [1, 6, 90])
def test_paged_nonfinite_values_stay_with_the_rows_that_see_them(bits, dtype, d, n):
    banner(f"paged nonfinite {bits} {dtype} {d} n={n}")
    x = Paged([n, n], [150, 300], 4, 2, d, dtype, bits, 32, seed=n + d)
    for m, k, v in zip(x.kv_lens, x.k, x.v):
        v[m - 1, 0, 3] = math.nan          # the last row's own
        v[m - n // 2 - 1, 1, 5] = math.inf  # seen by the later half
        v[m - n // 2 - 1, 1, 6] = -math.inf
        k[m - n // 3 - 1, 0, 2] = math.nan
        if n > 40:
            v[m - n + 20, 0, :] = math.inf
            v[m - n + 30, 0, 9] = -math.inf
    x.write()
    ref.check(x.run(), *x.expect(), "nonfinite")


def test_paged_window_leaves_nonfinite_values_behind():
    x = Paged([40], [400], 2, 1, 128, BF16, 16, 16, seed=5)
    x.v[0][320:350] = math.nan
    x.k[0][300:345] = math.inf
    x.write()
    got = x.run(window=30)
    want, bound = x.expect(window=30)
    assert torch.isfinite(want[-15:]).all() and not torch.isfinite(want[0]).all()
    ref.check(got, want, bound, "window")


def test_paged_large_scores():
    """Scores far apart: the running maximum moves by more than the exponent's range."""
    for dtype in (BF16, F16):
        x = Paged([1, 20], [700, 300], 4, 1, 128, dtype, 16, 64, seed=6, gain=40.0)
        ref.check(x.run(), *x.expect(), "large scores")


def test_paged_scale():
    x = Paged([3], [90], 4, 1, 64, BF16, 8, 16, seed=7)
    ref.check(x.run(scale=0.5), *x.expect(scale=0.5), "scale")


@pytest.mark.parametrize("n", [1, 33, 200])
def test_paged_strided_rows(n):
    d, hq, hkv = 128, 8, 2
    x = Paged([n, n], [n + 5, 400], hq, hkv, d, BF16, 16, 16, seed=8)
    want = x.run()
    qkv = torch.full((2 * n, (hq + 2 * hkv) * d), math.nan, dtype=BF16, device="cuda")
    q = ex.split_heads(qkv, hq, hkv, d)[0]
    q.copy_(x.q)
    assert same_bits(x.run(q=q), want)
    out = torch.zeros(hq, 2 * n, d + 8, dtype=BF16, device="cuda")
    got = x.run(out=out[:, :, :d].transpose(0, 1))
    assert same_bits(got, want) and not out[:, :, d:].any()


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_paged_long_context(bits):
    """Enough keys that one sequence is split into many parts, beside short ones."""
    banner(f"paged long {bits}")
    x = Paged([1, 2, 1], [30011, 9, 4097], 8, 1, 128, BF16, bits, 128, seed=9)
    ref.check(x.run(), *x.expect(), "long")
    ref.check(x.run(window=9001), *x.expect(window=9001), "long, window")
    first = x.run()
    for _ in range(3):
        assert same_bits(x.run(), first)


def test_paged_long_chunk():
    x = Paged([24, 100], [12345, 5000], 8, 1, 64, F16, 8, 64, seed=10)
    ref.check(x.run(), *x.expect(), "long chunk")


def test_paged_cache_past_four_gigabytes():
    pages, page, heads, d = 5200, 256, 8, 256
    cache = ex.KvCache.empty(pages, page, heads, d, 16, BF16)
    g = torch.Generator().manual_seed(11)
    k, v, q = (normal(g, (300, heads, d), BF16) for _ in range(3))
    table = torch.tensor([[pages - 1, 4100]], dtype=torch.int32)
    at = torch.arange(300)
    ex.cache_write(cache, k.cuda(), v.cuda(), (table[0, at // page].long() * page + at % page).int().cuda())
    for n in (1, 90):
        got = ex.paged_attention(cache, q[:n].cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                                 torch.tensor([300], dtype=torch.int32).cuda(), table.cuda())
        o, b = ref.attend(q[:n].double(), k.double(), v.double(), ref.mask(n, 300), d ** -0.5, BF16)
        ref.check(got, o, b, f"far pages, {n} rows")


# ------------------------------------------------------------------- prompts

class Packed:
    def __init__(self, lens, hq, hkv, d, dtype, seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        t = sum(lens)
        self.lens, self.dtype = lens, dtype
        self.q, self.k, self.v = normal(g, (t, hq, d), dtype, gain), normal(g, (t, hkv, d), dtype), normal(g, (t, hkv, d), dtype)
        self.cu = torch.tensor([0] + lens).cumsum(0).int()

    def run(self, **kw):
        return ex.prompt_attention(self.q.cuda(), self.k.cuda(), self.v.cuda(), self.cu.cuda(), **kw)

    def expect(self, causal=True, window=0):
        out, bound = [], []
        for i, n in enumerate(self.lens):
            a, b = int(self.cu[i]), int(self.cu[i + 1])
            o, e = ref.attend(self.q[a:b].double(), self.k[a:b].double(), self.v[a:b].double(),
                              ref.mask(n, n, causal, window), self.q.shape[-1] ** -0.5, self.dtype)
            out.append(o)
            bound.append(e)
        return torch.cat(out), torch.cat(bound)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2, 0, 1, 3], [31, 33, 64], [127, 129, 65], [400, 7]])
def test_prompt(lens, d, dtype):
    banner(f"prompt {lens} {d} {dtype}")
    x = Packed(lens, 6, 2, d, dtype, seed=d + len(lens))
    ref.check(x.run(), *x.expect(), "causal")
    ref.check(x.run(causal=False), *x.expect(causal=False), "not causal")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (7, 1), (12, 1), (24, 2)])
def test_prompt_groups(hq, hkv):
    banner(f"prompt groups {hq}/{hkv}")
    x = Packed([5, 150, 61], hq, hkv, 128, BF16, seed=hq)
    ref.check(x.run(), *x.expect(), f"{hq}/{hkv}")


@pytest.mark.parametrize("window", [1, 16, 63, 64, 65, 129, 500])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_window(window, d):
    x = Packed([300, 90], 4, 2, d, BF16, seed=window)
    ref.check(x.run(window=window), *x.expect(window=window), f"window {window}")


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16), (256, BF16)])
def test_prompt_nonfinite_values_stay_with_the_rows_that_see_them(d, dtype):
    x = Packed([200, 100], 4, 2, d, dtype, seed=d)
    x.v[50, 0, 3] = math.nan
    x.v[60, 1, 4], x.v[70, 1, 4] = math.inf, -math.inf
    x.v[150, :, :] = math.inf
    x.k[130, 0, 1] = math.nan
    x.k[250, 1, 2] = math.inf
    x.q[20, 1, 0] = math.nan
    x.v[299, 0, 7] = -math.inf
    ref.check(x.run(), *x.expect(), "nonfinite")


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (128, F16), (256, F16)])
def test_prompt_large_scores(d, dtype):
    x = Packed([260, 40], 4, 1, d, dtype, seed=d, gain=30.0)
    ref.check(x.run(), *x.expect(), "large scores")


def test_prompt_reads_views_of_one_projection():
    n, hq, hkv, d = 300, 8, 2, 128
    x = Packed([n], hq, hkv, d, BF16, seed=4)
    qkv = torch.cat([t.flatten(1) for t in (x.q, x.k, x.v)], 1).cuda()
    q, k, v = ex.split_heads(qkv, hq, hkv, d)
    want = x.run()
    assert same_bits(ex.prompt_attention(q, k, v, x.cu.cuda()), want)
    out = torch.zeros(n, 2 * hq, d, dtype=BF16, device="cuda")
    ex.prompt_attention(q, k, v, x.cu.cuda(), out=out[:, ::2])
    assert same_bits(out[:, ::2], want) and not out[:, 1::2].any()
    # one head's keys and values read as several
    k1, v1 = x.k[:, :1].cuda(), x.v[:, :1].cuda()
    wide = ex.prompt_attention(x.q.cuda(), k1.expand(n, 4, d), v1.expand(n, 4, d), x.cu.cuda())
    assert wide.shape == want.shape
    ref.check(wide, *ref.attend(x.q.double(), x.k[:, :1].double(), x.v[:, :1].double(), ref.mask(n, n), d ** -0.5, BF16),
              "expanded heads")


def test_prompt_and_cache_agree():
    """A prompt attended to directly and over a 16-bit cache of its keys: both within the bound."""
    n = 260
    x = Packed([n], 8, 2, 128, BF16, seed=12)
    cache = ex.KvCache.empty(6, 64, 2, 128, 16, BF16)
    ex.cache_write(cache, x.k.cuda(), x.v.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    got = ex.paged_attention(cache, x.q.cuda(), x.cu.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                             torch.arange(5, dtype=torch.int32, device="cuda")[None])
    want, bound = x.expect()
    ref.check(got, want, bound, "cache")
    ref.check(x.run(), want, bound, "direct")


@pytest.mark.parametrize("n", [3, 150])
def test_rows_past_32_bit_offsets(n):
    """Queries and results whose last rows are more than 2^32 bytes after their first: the same bits as dense ones."""
    hq, hkv, d = 8, 2, 64
    stride = -(-(2 ** 31 + 2 ** 20) // (n - 1)) // 8 * 8 + 8
    x = Packed([n], hq, hkv, d, BF16, seed=15)
    want = x.run()
    far = [torch.empty((n - 1) * stride + hq * d, dtype=BF16, device="cuda").as_strided((n, hq, d), (stride, d, 1))
           for _ in range(2)]
    assert (n - 1) * stride * 2 > 2 ** 32
    far[0].copy_(x.q)
    got = ex.prompt_attention(far[0], x.k.cuda(), x.v.cuda(), x.cu.cuda(), out=far[1])
    assert got is far[1] and same_bits(got, want)
    cache = ex.KvCache.empty(3, 64, hkv, d, 16, BF16)
    ex.cache_write(cache, x.k.cuda(), x.v.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    lens, table = torch.tensor([n], dtype=torch.int32).cuda(), torch.arange(3, dtype=torch.int32, device="cuda")[None]
    want = ex.paged_attention(cache, x.q.cuda(), x.cu.cuda(), lens, table)
    assert same_bits(ex.paged_attention(cache, far[0], x.cu.cuda(), lens, table, out=far[1]), want)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 100])
def test_a_nonfinite_query_row_stays_alone(n, d):
    x = Packed([n, 40], 6, 2, d, BF16, seed=16)
    want = x.run()
    x.q[1, 4] = math.nan
    x.q[2, 0, 7] = math.inf
    got = x.run()
    assert got[1, 4].isnan().all() and not got[2, 0].isfinite().all()
    keep = torch.ones(n + 40, 6, dtype=torch.bool)
    keep[1, 4] = keep[2, 0] = False
    assert same_bits(got.cpu()[keep], want.cpu()[keep])


def test_no_tokens():
    empty = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ex.prompt_attention(empty, empty, empty, cu).shape == (0, 4, 64)
    cache = ex.KvCache.empty(1, 16, 4, 64, 16, BF16)
    got = ex.paged_attention(cache, empty, cu, torch.zeros(2, dtype=torch.int32, device="cuda"),
                             torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    assert got.shape == (0, 4, 64)


def test_lengths_that_do_not_fit_stay_inside_the_buffers():
    """Offsets past the rows, falling ones and negative lengths: other sequences are right, nothing faults."""
    x = Paged([4, 4, 4], [50, 60, 70], 4, 2, 64, BF16, 16, 16, seed=13)
    want = x.run()
    kv = torch.tensor([50, -5, 70], dtype=torch.int32).cuda()
    got = ex.paged_attention(x.cache, x.q.cuda(), x.cu.cuda(), kv, x.table.cuda())
    assert same_bits(got[:4], want[:4]) and same_bits(got[8:], want[8:]) and not got[4:8].any()
    cu = torch.tensor([0, 4, 2, 9000], dtype=torch.int32).cuda()
    got = ex.paged_attention(x.cache, x.q.cuda(), cu, torch.tensor(x.kv_lens, dtype=torch.int32).cuda(), x.table.cuda())
    assert same_bits(got[:2], want[:2])


def test_on_another_stream_and_in_a_graph():
    x = Paged([1, 1, 2], [9000, 50, 700], 8, 2, 128, BF16, 8, 64, seed=14)
    q, cu, table = x.q.cuda(), x.cu.cuda(), x.table.cuda()
    kv = torch.tensor(x.kv_lens, dtype=torch.int32).cuda()
    want = x.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ex.paged_attention(x.cache, q, cu, kv, table)
    side.synchronize()
    assert same_bits(got, want)
    r = ex.Rope.make(128, 10000.0, 100)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    kvrow = torch.zeros(4, 2, 128, dtype=BF16, device="cuda")
    out, q2 = torch.empty_like(q), torch.empty_like(q)
    with torch.cuda.stream(side):
        ex.reserve_workspace(ex.attention_workspace_bytes(3, 4, 8, 2, 128))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ex.rope_cache_write(x.cache, r, pos, slots, q, kvrow, kvrow, q_out=q2)
        ex.paged_attention(x.cache, q2, cu, kv, table, out=out)
    for i in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want), f"replay {i}"
        assert same_bits(x.run(), want)
        kv.sub_(1).add_(1)  # the program's own work between replays
