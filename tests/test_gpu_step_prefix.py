"""GPU: attention of sequences that share prefixes, against the definition in
64 bits (attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
import test_gpu_attention as base
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
same_bits, normal = base.same_bits, base.normal


def widened(cache, table):
    """The page table as a part of one with so many columns that a call for two sequences and one group shares."""
    row = cache.head_dim * cache.bits // 8 + (cache.head_dim // 32 if cache.bits < 16 else 0)
    columns = int(200e6 / (cache.page_size * cache.heads * 2 * row)) + 1
    big = torch.full((table.shape[0], max(columns, table.shape[1])), -1, dtype=torch.int32, device="cuda")
    big[:, :table.shape[1]] = table
    return big


class Shared:
    """Groups of sequences: groups[g] = (prefix keys, [(new tokens, keys after the prefix), ...]).  Shared keys lie in the
    same pages, whole ones; the rest of them begins every sequence's own pages.  A key count below zero shortens the
    sequence into the prefix.  Unused pages and slots hold NaN."""

    def __init__(self, groups, hq, hkv, d, dtype, bits, page, seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.dtype, self.groups = page, dtype, groups
        seqs = [(i, q, p + own) for i, (p, members) in enumerate(groups) for q, own in members]
        self.q_lens, self.kv_lens = [s[1] for s in seqs], [s[2] for s in seqs]
        each = [p // page for p, _ in groups]  # whole pages
        self.shared = [e * page for e in each]
        per = [max(0, -(-n // page) - each[i]) for i, _, n in seqs]
        pages = sum(each) + sum(per) + 3
        order, at = torch.randperm(pages, generator=g).int(), sum(each)
        starts = torch.tensor([0] + each).cumsum(0).tolist()
        self.table = torch.full((len(seqs), max([each[i] + n for (i, _, _), n in zip(seqs, per)]) + 1), -1, dtype=torch.int32)
        for s, ((i, _, _), n) in enumerate(zip(seqs, per)):
            self.table[s, :each[i]] = order[starts[i]:starts[i] + each[i]]
            self.table[s, each[i]:each[i] + n] = order[at:at + n]
            at += n
        self.cache = ex.KvCache.empty(pages, page, hkv, d, bits, dtype)
        nan = torch.full((pages * page, hkv, d), math.nan, dtype=dtype, device="cuda")
        ex.cache_write(self.cache, nan, nan, torch.arange(pages * page, dtype=torch.int32, device="cuda"))
        front = [[normal(g, (n, hkv, d), dtype, s) for s in (gain, 1.0)] for n in self.shared]
        self.k, self.v = [], []
        for i, _, n in seqs:
            for to, f, s in ((self.k, front[i][0], gain), (self.v, front[i][1], 1.0)):
                to.append(torch.cat((f, normal(g, (max(0, n - len(f)), hkv, d), dtype, s)))[:n])
        self.front = front
        self.q = normal(g, (sum(self.q_lens), hq, d), dtype)
        self.cu = torch.tensor([0] + self.q_lens).cumsum(0).int()
        self.group_cu = torch.tensor([0] + [len(m) for _, m in groups]).cumsum(0).int()
        self.prefix = torch.tensor([p for p, _ in groups], dtype=torch.int32)
        self.write()

    def write(self):
        pos = lambda n: torch.arange(n)  # noqa: E731
        for s, n in enumerate(self.kv_lens):
            if n:
                slots = self.table[s, pos(n) // self.page].long() * self.page + pos(n) % self.page
                ex.cache_write(self.cache, self.k[s].cuda(), self.v[s].cuda(), slots.int().cuda())
        for g, n in enumerate(self.shared):  # whole, also where all sequences are shorter
            s = int(self.group_cu[g])
            if n and self.group_cu[g + 1] > s:
                slots = self.table[s, pos(n) // self.page].long() * self.page + pos(n) % self.page
                ex.cache_write(self.cache, self.front[g][0].cuda(), self.front[g][1].cuda(), slots.int().cuda())

    def args(self, wide=True):
        """Arguments with a page table of wide rows, by whose size the call goes for the shared passes, or as it is."""
        table = self.table.cuda()
        return (self.cache, self.q.cuda(), self.cu.cuda(), torch.tensor(self.kv_lens, dtype=torch.int32).cuda(),
                widened(self.cache, table) if wide else table)

    def run(self, group_cu=None, prefix=None, **kw):
        ints = lambda x, y: (x if y is None else torch.tensor(y, dtype=torch.int32)).cuda()  # noqa: E731
        # what is shared in earnest: whole pages
        shared = torch.tensor(self.shared, dtype=torch.int32)
        return ex.prefix_attention(*self.args(kw.pop("wide", True)), ints(self.group_cu, group_cu), ints(shared, prefix), **kw)

    def expect(self, scale=None):
        bits, d = self.cache.bits, self.q.shape[-1]
        out, bound = [], []
        for i, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            seen = ref.mask(n, m, True, 0, self.table[i], self.page, self.cache.pages)
            o, b = ref.attend(self.q[self.cu[i]:self.cu[i + 1]].double(), ref.quantise(self.k[i], bits),
                              ref.quantise(self.v[i], bits), seen, d ** -0.5 if scale is None else scale, self.dtype)
            out.append(o)
            bound.append(b)
        return torch.cat(out), torch.cat(bound)

    def check(self, what="", **kw):
        want = self.expect()
        ref.check(self.run(**kw), *want, what or "attention")
        # and the call that its sizes leave to the plain kernels
        ref.check(self.run(wide=False, **kw), *want, "narrow")
        return want


@pytest.mark.parametrize("bits,dtype,d", base.FORMATS)
@pytest.mark.parametrize("members", [2, 7, 40])
def test_one_token(bits, dtype, d, members):
    banner(f"shared prefix, {members} sequences, {bits} bits {dtype} d={d}")
    x = Shared([(150, [(1, 1 + 13 * i % 70) for i in range(members)])], 4, 2, d, dtype, bits, 16, seed=1)
    x.check()


@pytest.mark.parametrize("bits,dtype,d", base.FORMATS)
def test_several_tokens_in_several_groups(bits, dtype, d):
    """Own keys and shared keys on the kernel for many rows, sequences without new tokens, a group of one, an empty one."""
    x = Shared([(96, [(70, 90), (0, 5), (33, 40)]), (200, [(50, 77)]), (64, []), (330, [(1, 1), (80, 80), (2, 300)])], 6, 2, d, dtype,
               bits, 32, seed=2)
    x.check()


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("prefix", [0, 15, 16, 31, 32, 33, 64, 127, 128, 129, 255, 256, 500])
def test_lengths_of_the_prefix(prefix, page):
    x = Shared([(prefix, [(1, 3), (2, 60), (1, 1)]), (prefix // 2, [(3, 3), (1, 100)])], 4, 1, 128, F16, 16, page, seed=prefix)
    x.check()


def test_lengths_that_are_no_pages():
    """Sequences that are alike to their end may name any length."""
    x = Shared([(256, [(1, 0), (2, 0), (1, 0)])], 4, 2, 64, BF16, 8, 64, seed=3)
    want = x.expect()
    for n in (1, 31, 33, 100, 200, 254, 255, 256, 257, 10000, 2 ** 31 - 1, 0, -1, -2 ** 31):
        ref.check(x.run(prefix=[n]), *want, f"prefix {n}")


def test_sequences_that_end_within_the_prefix():
    x = Shared([(320, [(1, 50), (1, -100), (4, 9), (0, -310), (2, -30)])], 4, 2, 128, BF16, 16, 16, seed=4)
    x.check()
    x = Shared([(320, [(1, 50), (5, -318)])], 4, 2, 128, BF16, 16, 16, seed=5)  # more new tokens than keys
    x.check()


@pytest.mark.parametrize("hq,hkv,members,n", [(1, 1, 3, 1), (8, 8, 5, 2), (12, 2, 20, 1), (16, 1, 9, 3), (3, 3, 200, 1), (32, 4, 70, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_heads_and_members(hq, hkv, members, n, d):
    x = Shared([(100, [(n, n + i % 37) for i in range(members)])], hq, hkv, d, BF16, 8, 16, seed=6)
    x.check()


@pytest.mark.parametrize("batch", [2, 63, 64, 65, 255, 256, 257])
def test_groups_of_every_size_by_either_form(batch):
    """Up to 255 sequences the kernels of the shared keys find the groups themselves: one group, groups of two, and
    groups with sequences that have no new tokens."""
    one = Shared([(64, [(1, 1 + i % 20) for i in range(batch)])], 2, 1, 64, BF16, 8, 16, seed=26)
    one.check()
    pairs = Shared([(32, [(1, 1 + i % 9), (i % 2, 5)]) for i in range(batch // 2)] + [(32, [])], 2, 1, 64, BF16, 8, 16, seed=27)
    pairs.check()


@pytest.mark.parametrize("bits,dtype,d", base.FORMATS)
@pytest.mark.parametrize("n", [1, 3])
def test_the_smallest_groups(n, bits, dtype, d):
    """Two sequences in one group, with one beside them, with sequences of no group (more sequences than groups: the
    shared passes take them; as many of both are one plain launch)."""
    for groups in ([(64, [(n, n), (n, n + 5)])], [(96, [(n, n + 40), (1, 2)]), (32, [(n, n + 7)])],
                   [(32, [(0, 4), (n, n + 9), (2, 3)]), (48, [])]):
        x = Shared(groups, 4, 2, d, dtype, bits, 16, seed=32)
        assert len(x.kv_lens) > len(x.groups)
        want = x.check()
        ref.check(x.run(group_cu=[0, 2], prefix=[x.shared[0]]), *want, "the first two")
        ref.check(x.run(group_cu=[1, len(x.kv_lens)], prefix=[0]), *want, "a group that shares nothing")


@pytest.mark.parametrize("n", [128, 129])
def test_chunks_up_to_and_past_what_is_shared(n):
    """512 rows of a sequence on each key/value head are the most that the shared passes take."""
    x = Shared([(224, [(n, n + 30), (n, n + 1)])], 8, 2, 128, BF16, 8, 16, seed=30)
    x.check()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hundreds_of_sequences_with_tiles_of_rows(d):
    """Own keys by the kernel of many rows, one and two tiles of a sequence, found among 270 sequences."""
    x = Shared([(48, [((0, 20, 37, 23)[i % 4], 40 + i % 11) for i in range(200)]), (16, [(21, 30 + i) for i in range(70)])], 8, 2, d,
               BF16, 8, 16, seed=31)
    x.check()


def test_thousands_of_sequences_some_without_new_tokens():
    """The own keys' rows of a sequence are found among 4200 by three looks at 64."""
    x = Shared([(16, [((i + j) % 3, 2 + (i * j) % 7) for j in range(3)]) for i in range(1400)], 2, 1, 64, BF16, 8, 16, seed=28)
    x.check()


@pytest.mark.parametrize("others", [0, 260])
def test_ended_sequences_whose_pages_are_gone(others):
    """A server's slots that hold no request: no new tokens, and a row of the page table without pages or with others'."""
    x = Shared([(96, [(0, 5), (1, 9), (0, 3), (2, 60), (1, 1), (0, 7)]), (64, [(0, 1), (0, 2)]), (48, [(0, 1), (1, 9), (3, 3)]),
                (32, [(0, 1), (1, 9)])] + [(16, [(1, 2)] * others)] * (others > 0), 4, 2, 64, BF16, 8, 16, seed=29)
    for s in (0, 2, 5, 6, 8, 11):
        x.table[s] = -1 if s % 2 == 0 else 1
        x.kv_lens[s] = 0 if s % 4 == 0 else 40
    x.check()


def test_more_sequences_than_a_workgroup_looks_at_together():
    x = Shared([(48, [(1, 1 + i % 20) for i in range(300)]), (32, [(1, 2)] * 280)], 2, 1, 64, BF16, 16, 16, seed=7)
    x.check()


@pytest.mark.parametrize("bits,d", [(16, 128), (8, 64), (4, 256)])
@pytest.mark.parametrize("n,members", [(1, 3), (1, 60), (40, 3)])
def test_long_prefixes_and_long_own_keys_in_parts(bits, d, n, members):
    x = Shared([(9600, [(n, n + (3000 if i == 1 else 9 * i)) for i in range(members)])], 4, 1, d, BF16, bits, 64, seed=8)
    got = x.run().cpu()
    pick = sorted({0, n - 1, n, 2 * n - 1, len(x.q) - 1})
    for r in pick:
        s = int((x.cu <= r).sum()) - 1
        m = x.kv_lens[s] - x.q_lens[s] + r - int(x.cu[s]) + 1
        seen = torch.ones(1, m, dtype=torch.bool)
        want = ref.attend(x.q[r:r + 1].double(), ref.quantise(x.k[s][:m], bits), ref.quantise(x.v[s][:m], bits), seen, d ** -0.5, BF16)
        ref.check(got[r:r + 1], *want, f"row {r}")
    plain = ex.paged_attention(*x.args()).double().cpu()
    # both are within a rounding of probabilities and results of the same numbers
    assert (got.double() - plain).abs().max() <= 4 * 2.0 ** -8 * plain.abs().max()


def test_holes():
    x = Shared([(160, [(2, 60), (1, 70), (3, 80)]), (64, [(1, 4), (1, 5)])], 4, 2, 64, F16, 16, 16, seed=9)
    x.table[:3, 2:4] = -1                # shared pages
    x.table[1, 11] = -1                  # one of a sequence's own
    x.table[2, 10:] = x.cache.pages      # all of a sequence's own
    x.table[3:, :] = -1                  # everything of a group
    x.check()
    assert not x.run()[6:].any()
    kv, cu = torch.tensor(x.kv_lens, dtype=torch.int32).cuda(), x.cu.cuda()
    x.table[:, 3:] = -1  # a table narrower than the prefix
    ref.check(x.run(), *x.expect(), "shared pages after the third gone")
    got = ex.prefix_attention(x.cache, x.q.cuda(), cu, kv, x.table[:, :3].contiguous().cuda(), x.group_cu.cuda(), x.prefix.cuda())
    ref.check(got, *x.expect(), "narrow")
    none = torch.zeros(5, 0, dtype=torch.int32, device="cuda")
    assert not ex.prefix_attention(x.cache, x.q.cuda(), cu, kv, none, x.group_cu.cuda(), x.prefix.cuda()).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("members", [3, 50])
def test_values_that_are_not_finite(dtype, members):
    """Own ones stay with their sequence, shared ones reach all; a query row with NaN stays alone."""
    x = Shared([(128, [(1, 20 + i % 5) for i in range(members)])], 4, 2, 128, dtype, 16, 16, seed=10)
    x.v[1][140, 0, 3] = math.inf
    x.k[2][145, 1] = math.nan
    x.write()
    x.check()
    got = x.run().cpu()
    assert torch.isinf(got[1, :2, 3]).all() and torch.isfinite(got[0]).all()
    for s in range(members):
        x.v[s][7, 1, 5] = -math.inf
    x.front[0][1][7, 1, 5] = -math.inf
    x.k[2][145, 1] = 1.0
    x.q[0, 0, 0] = math.nan
    x.write()
    got = x.run().cpu()
    assert torch.isnan(got[0, 0]).all() and torch.isinf(got[0, 2:, 5]).all() and torch.isinf(got[1:, 2:, 5]).all()
    assert torch.isfinite(got[1:, :2, :3]).all() and torch.isfinite(got[0, 1]).all()


def test_large_scores_and_scale():
    x = Shared([(200, [(1, 30), (2, 40), (1, 9)])], 4, 2, 64, BF16, 16, 16, seed=11, gain=30.0)
    x.check()
    ref.check(x.run(scale=0.01), *x.expect(0.01), "scale")


def test_groups_that_do_not_fit():
    """Falling offsets and offsets past the sequences: the sequences of the groups that are left are right."""
    x = Shared([(160, [(1, 20), (2, 30), (1, 40), (2, 9)])], 4, 2, 64, BF16, 8, 16, seed=12)
    want = x.expect()
    for cu in ([0, 4], [1, 3], [2, 2], [-7, 900], [3, 0], [2 ** 31 - 1, 4], [0, 0]):
        ref.check(x.run(group_cu=cu), *want, f"groups {cu}")
    for cu, prefix in (([0, 3, 1, 4], [160, 160, 32]), ([1, 1, 2, 4], [160, 100, 160]), ([0, 2, 4], [-5, 160]), ([0], [])):
        ref.check(x.run(group_cu=cu, prefix=prefix), *want, f"groups {cu}")


def test_lengths_that_do_not_fit_stay_inside_the_buffers():
    x = Shared([(160, [(4, 20), (4, 30), (4, 40)])], 4, 2, 64, BF16, 16, 16, seed=13)
    want = x.run()
    cache, q, cu, kv, table = x.args()
    groups, shared = x.group_cu.cuda(), torch.tensor(x.shared, dtype=torch.int32).cuda()
    kv2 = torch.tensor([180, -5, 200], dtype=torch.int32).cuda()
    got = ex.prefix_attention(cache, q, cu, kv2, table, groups, shared)
    plain = ex.paged_attention(cache, q, cu, kv2, table)
    assert not got[4:8].any() and (got.double() - plain.double()).abs().max() <= 4 * 2.0 ** -8 * plain.double().abs().max()
    cu2 = torch.tensor([0, 4, 2, 9000], dtype=torch.int32).cuda()
    got = ex.prefix_attention(cache, q, cu2, kv, table, groups, shared)
    plain = ex.paged_attention(cache, q, cu2, kv, table)
    assert (got[:2].double() - plain[:2].double()).abs().max() <= 4 * 2.0 ** -8 * plain[:2].double().abs().max()
    assert (got[:4].double() - want[:4].double()).abs().max() <= 4 * 2.0 ** -8 * want.double().abs().max()


@pytest.mark.parametrize("n", [1, 40])
def test_strided_rows_and_in_place(n):
    x = Shared([(160, [(n, n + 20), (n, n + 30)])], 4, 2, 64, F16, 8, 16, seed=14)
    want = x.run()
    wide = torch.zeros(2 * n, 9, 80, dtype=F16, device="cuda")
    view = wide[:, 2:6, 8:72]
    view.copy_(x.q.cuda())
    cache, _, cu, kv, table = x.args()
    more = (x.group_cu.cuda(), torch.tensor(x.shared, dtype=torch.int32).cuda())
    assert same_bits(ex.prefix_attention(cache, view, cu, kv, table, *more), want)
    got = ex.prefix_attention(cache, view, cu, kv, table, *more, out=view)
    assert got is view and same_bits(view, want)
    wide[:, 2:6, 8:72] = 0
    assert not wide.any()


def test_no_tokens():
    cache = ex.KvCache.empty(1, 16, 4, 64, 16, BF16)
    empty = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert ex.prefix_attention(cache, empty, z(3), z(2), z(2, 1), z(2), z(1)).shape == (0, 4, 64)


def test_graphs_that_share_a_workspace_and_lengths_that_change():
    """Two captured calls on one stream, replayed in turn with eager ones between, the second's lengths changing."""
    x = Shared([(640, [(1, 50 + i) for i in range(9)])], 8, 2, 128, BF16, 8, 64, seed=15)
    y = Shared([(1280, [(2, 90), (1, 3000), (3, 7)]), (64, [(1, 1), (1, 2)])], 8, 2, 128, BF16, 8, 64, seed=16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = []
    for z in (x, y):
        cache, q, cu, kv, table = z.args()
        calls.append((cache, q, cu, kv, table, z.group_cu.cuda(), torch.tensor(z.shared, dtype=torch.int32).cuda()))
    with torch.cuda.stream(side):
        for z in (x, y):
            ex.reserve_workspace(ex.prefix_attention_workspace_bytes(len(z.kv_lens), len(z.q), len(z.groups), 8, 2, 128))
    torch.cuda.synchronize()
    outs, graphs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(ex.prefix_attention(*c))
    for i in range(3):
        for j, (g, o, c) in enumerate(zip(graphs, outs, calls)):
            o.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
                eager = ex.prefix_attention(*c)
            torch.cuda.synchronize()
            assert same_bits(o, eager), f"graph {j}, replay {i}"
        calls[1][3].sub_(1)  # every sequence a key shorter


def test_cache_past_four_gigabytes():
    """Pages whose bytes lie past 2^32."""
    cache = ex.KvCache.empty(20000, 256, 8, 64, 16, BF16)  # 5.2 GB each of keys and values
    g = torch.Generator().manual_seed(17)
    k, v = (normal(g, (3, 300, 8, 64), BF16) for _ in range(2))
    k[:, :256], v[:, :256] = k[:1, :256], v[:1, :256]
    table = torch.tensor([[19999, 19998], [19999, 19997], [19999, 3]], dtype=torch.int32).cuda()
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    for s in range(3):
        ex.cache_write(cache, k[s].cuda(), v[s].cuda(), cache.slots(table, torch.full_like(pos, s), pos))
    table = widened(cache, table)
    for n in (1, 60):
        q = normal(g, (3 * n, 8, 64), BF16)
        ints = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        got = ex.prefix_attention(cache, q.cuda(), ints(0, n, 2 * n, 3 * n), ints(300, 300, 280 + n // 4), table, ints(0, 3), ints(256))
        for s, m in enumerate((300, 300, 280 + n // 4)):
            seen = ref.mask(n, m)
            ref.check(got[s * n:s * n + n], *ref.attend(q[s * n:s * n + n].double(), k[s, :m].double(), v[s, :m].double(), seen, 0.125,
                                                        BF16), f"sequence {s}")
