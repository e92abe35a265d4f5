"""GPU: attention with a window and first tokens that stay visible, over the
paged cache and over packed prompts, against the definition in 64 bits
(attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as ref
import attn_tile_cases as cases
import linear_exl3_input_amd as ex
import test_gpu_attention as base
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
same_bits = base.same_bits


def seen_of(q, kv, window, sinks, *table):
    gap = torch.arange(kv - q, kv)[:, None] - torch.arange(kv)
    return ref.mask(q, kv, True, 0, *table) & ((gap < window) | (torch.arange(kv) < sinks))


class Paged(base.Paged):
    def expect(self, window, sinks):
        bits, d = self.cache.bits, self.q.shape[-1]
        out, bound = [], []
        for i, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            seen = seen_of(n, m, window, sinks, self.table[i], self.page, self.cache.pages)
            o, b = ref.attend(self.q[self.cu[i]:self.cu[i + 1]].double(), ref.quantise(self.k[i], bits),
                              ref.quantise(self.v[i], bits), seen, d ** -0.5, self.dtype)
            out.append(o)
            bound.append(b)
        return torch.cat(out), torch.cat(bound)

    def check(self, window, sinks):
        ref.check(self.run(window=window, sinks=sinks), *self.expect(window, sinks), f"window {window}, sinks {sinks}")

    def free(self, window, sinks):
        """Takes from the table the pages that no row sees."""
        for i, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            first = max(0, m - n - window + 1)
            for j in range(self.table.shape[1]):
                if j * self.page >= sinks and (j + 1) * self.page <= first:
                    self.table[i, j] = -1


class Packed(base.Packed):
    def check(self, window, sinks):
        got = self.run(window=window, sinks=sinks)
        for i, n in enumerate(self.lens):
            a, b = int(self.cu[i]), int(self.cu[i + 1])
            want = ref.attend(self.q[a:b].double(), self.k[a:b].double(), self.v[a:b].double(), seen_of(n, n, window, sinks),
                              self.q.shape[-1] ** -0.5, self.dtype)
            ref.check(got[a:b], *want, f"sequence {i}, window {window}, sinks {sinks}")


@pytest.mark.parametrize("bits,dtype,d", base.FORMATS)
@pytest.mark.parametrize("freed", [False, True])
def test_one_token(bits, dtype, d, freed):
    banner(f"sinks, one token, {bits} bits {dtype} d={d} freed={freed}")
    x = Paged([1, 1, 1, 1], [700, 1, 5, 333], 4, 2, d, dtype, bits, 16, seed=1)
    for window, sinks in ((100, 4), (33, 70), (1, 1)) if not freed else ((100, 4),):
        if freed:
            x.free(window, sinks)
        x.check(window, sinks)


@pytest.mark.parametrize("bits,dtype,d", base.FORMATS)
@pytest.mark.parametrize("freed", [False, True])
def test_chunks(bits, dtype, d, freed):
    """On the kernel for many rows."""
    banner(f"sinks, chunks, {bits} bits {dtype} d={d} freed={freed}")
    x = Paged([70, 0, 150], [500, 40, 433], 6, 2, d, dtype, bits, 32, seed=2)
    window, sinks = (60, 9) if freed else (130, 40)
    if freed:
        x.free(window, sinks)
    x.check(window, sinks)


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 31), (31, 32), (32, 33), (33, 63), (64, 64), (65, 127), (100, 128), (128, 129),
                                          (20, 200), (300, 1), (340, 4), (600, 3), (2 ** 30, 2 ** 20), (7, 2 ** 20), (2 ** 30, 1), (250, 96)])
def test_windows_and_sinks(window, sinks, d, n):
    x = Paged([n, min(n, 7)], [n + 350, 7], 4, 1, d, F16, 16, 16, seed=window + sinks)
    x.check(window, sinks)


@pytest.mark.parametrize("bits,d", [(16, 128), (8, 64), (4, 256)])
@pytest.mark.parametrize("n", [1, 3, 100])
def test_parts(bits, d, n):
    """Windows and first tokens long enough to be split, the first tokens over several parts."""
    x = Paged([n, min(n, 2)], [9000, 6100], 4, 1, d, BF16, bits, 64, seed=3)
    for window, sinks in ((3000, 20), (1200, 2500), (4000, 4900)):
        x.check(window, sinks)


@pytest.mark.parametrize("n", [1, 80])
def test_holes_and_empty_rows(n):
    x = Paged([n, n], [n + 300, n + 200], 4, 2, 64, BF16, 8, 16, seed=4)
    x.table[0, 0] = -1                   # the first tokens
    x.table[0, 15:18] = -1               # some of the window
    x.table[1, :] = -1                   # all
    x.table[1, 5] = x.cache.pages        # none of the cache's
    x.check(100, 20)
    assert not x.run(window=100, sinks=20)[n:].any()


@pytest.mark.parametrize("n", [1, 80])
def test_table_ends_before_the_window_or_within_the_first_tokens(n):
    x = Paged([n], [n + 900], 4, 2, 64, F16, 16, 16, seed=5)
    kv = torch.tensor(x.kv_lens, dtype=torch.int32).cuda()
    whole = x.table.clone()
    for width in (1, 2, 3, 9, 50):
        x.table = whole.clone()
        x.table[:, width:] = -1
        got = ex.paged_attention(x.cache, x.q.cuda(), x.cu.cuda(), kv, whole[:, :width].contiguous().cuda(), window=50, sinks=37)
        ref.check(got, *x.expect(50, 37), f"width {width}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (256, 1), (64, 90), (128, 90), (256, 90)])
@pytest.mark.parametrize("bits", [16, 8])
def test_nonfinite_values_stay_with_the_rows_that_see_them(bits, dtype, d, n):
    x = Paged([n], [n + 260], 2, 1, d, dtype, bits, 16, seed=6)
    x.v[0][20:90, 0, 3] = math.inf      # between the first tokens and every window
    x.k[0][20:90, 0] = math.nan
    x.v[0][2, 0, 5] = math.inf          # a first token
    x.v[0][n + 200, 0, 7] = -math.inf   # seen by the rows up to it + window
    x.write()
    if bits == 16:
        x.check(70, 11)
    else:  # a block of 32 values with an infinity reads as NaN
        got = x.run(window=70, sinks=11).cpu()
        want, _ = x.expect(70, 11)
        assert torch.equal(torch.isnan(got), torch.isnan(want))


def test_few_keys_many_rows_and_lengths_that_do_not_fit():
    x = Paged([4, 90, 3], [2, 30, 0], 4, 2, 64, BF16, 16, 16, seed=7)  # more new tokens than keys
    x.check(3, 2)
    x = Paged([4, 4, 4], [50, 60, 70], 4, 2, 64, BF16, 16, 16, seed=8)
    want = x.run(window=20, sinks=5)
    kv = torch.tensor([50, -5, 70], dtype=torch.int32).cuda()
    got = ex.paged_attention(x.cache, x.q.cuda(), x.cu.cuda(), kv, x.table.cuda(), window=20, sinks=5)
    assert same_bits(got[:4], want[:4]) and same_bits(got[8:], want[8:]) and not got[4:8].any()


def test_no_window_or_no_sinks_are_the_plain_calls():
    x = Paged([3, 70], [200, 300], 4, 2, 128, BF16, 8, 16, seed=9)
    assert same_bits(x.run(sinks=4), x.run()) and same_bits(x.run(window=40, sinks=0), x.run(window=40))
    y = Packed([100, 33], 4, 2, 128, BF16, seed=9)
    assert same_bits(y.run(sinks=4), y.run()) and same_bits(y.run(causal=False, sinks=4), y.run(causal=False))
    with pytest.raises(ValueError, match="sinks=-1"):
        x.run(window=4, sinks=-1)
    with pytest.raises(ValueError, match="sinks="):
        y.run(sinks=2 ** 20 + 1)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2, 0, 1, 3], [31, 33, 64], [127, 129, 65], [400, 7]])
def test_prompts(lens, d, dtype):
    banner(f"sinks, prompts {lens} d={d} {dtype}")
    x = Packed(lens, 6, 2, d, dtype, seed=10)
    for window, sinks in ((1, 1), (40, 4), (33, 130), (100, 64)):
        x.check(window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_in_parts_and_in_whole_tiles(d):
    """The sizes of attn_tile_cases, whose kernel is checked without a GPU; rows at chosen places."""
    for c in (cases.PROMPTS[d], cases.FULL[d]):
        if c["prompt"]:
            x = Packed(c["q_lens"], c["hq"], c["hkv"], d, BF16, seed=11)
            got = x.run(window=1500, sinks=77)
            at = 0
            for i, n in enumerate(c["q_lens"]):
                pick = torch.tensor(sorted({0, 1, 76, 77, n // 2, min(n - 1, 1577), min(n - 1, 1700), n - 2, n - 1}))
                seen = seen_of(n, n, 1500, 77)[pick]
                k, v = (t[at:at + n].double() for t in (x.k, x.v))
                ref.check(got[at + pick], *ref.attend(x.q[at + pick].double(), k, v, seen, d ** -0.5, BF16), f"prompt {i}")
                at += n
        else:
            x = Paged(c["q_lens"], c["kv_lens"], c["hq"], c["hkv"], d, BF16, 8, 256, seed=12)
            got = x.run(window=500, sinks=130)
            at = 0
            for i, (n, m) in enumerate(zip(c["q_lens"], c["kv_lens"])):
                pick = torch.tensor([0, n // 3, n - 1])
                seen = seen_of(n, m, 500, 130)[pick]
                h = torch.arange(4)  # the query heads of key/value head 0
                k, v = (ref.quantise(t[i][:, :1], 8) for t in (x.k, x.v))
                ref.check(got[at + pick][:, h], *ref.attend(x.q[at + pick][:, h].double(), k, v, seen, d ** -0.5, BF16), f"chunk {i}")
                at += n


def test_on_another_stream_and_in_a_graph():
    x = Paged([1, 1, 2], [9000, 50, 700], 8, 2, 128, BF16, 8, 64, seed=14)
    q, cu, table = x.q.cuda(), x.cu.cuda(), x.table.cuda()
    kv = torch.tensor(x.kv_lens, dtype=torch.int32).cuda()
    want = x.run(window=5000, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ex.paged_attention(x.cache, q, cu, kv, table, window=5000, sinks=4)
        ex.reserve_workspace(ex.attention_workspace_bytes(3, 4, 8, 2, 128))
    side.synchronize()
    assert same_bits(got, want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ex.paged_attention(x.cache, q, cu, kv, table, out=out, window=5000, sinks=4)
    for i in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want) and same_bits(x.run(window=5000, sinks=4), want), f"replay {i}"


def test_cache_past_four_gigabytes():
    """Pages whose bytes lie past 2^32."""
    cache = ex.KvCache.empty(20000, 256, 8, 64, 16, BF16)  # 5.2 GB each of keys and values
    g = torch.Generator().manual_seed(15)
    k, v = (base.normal(g, (300, 8, 64), BF16) for _ in range(2))
    table = torch.tensor([[19999, 19998]], dtype=torch.int32).cuda()
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    ex.cache_write(cache, k.cuda(), v.cuda(), cache.slots(table, torch.zeros_like(pos), pos))
    for n in (1, 150):
        q = base.normal(g, (n, 8, 64), BF16)
        got = ex.paged_attention(cache, q.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                                 torch.tensor([300], dtype=torch.int32).cuda(), table, window=40, sinks=3)
        ref.check(got, *ref.attend(q.double(), k.double(), v.double(), seen_of(n, 300, 40, 3), 0.125, BF16), f"{n} rows")
