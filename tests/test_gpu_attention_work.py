"""GPU: how the attention calls find their work: offsets that no caller should
pass, many sequences."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(seed, shape, dtype=BF16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def counters():
    return ex._workspaces[ex.workspace_key()][:ex.COUNTER_BYTES].view(torch.int32)


def test_falling_offsets_leave_the_counters_clear():
    """Five times the same 2000 rows: taken at their word they would make 378 work items a head (4 x 63 tiles, and 63 of
    the last sequence's 100000 keys in two parts) where the launch has 327, so that parts would be missing and their
    counters stay set.  Afterwards the same stream's calls are right."""
    banner("falling offsets")
    page, hq, hkv, d, n, long = 1024, 32, 8, 128, 2000, 100000
    cache = ex.KvCache.empty(2, page, hkv, d)
    k, v = normal(1, (2 * page, hkv, d)).cuda(), normal(2, (2 * page, hkv, d)).cuda()
    ex.cache_write(cache, k, v, torch.arange(2 * page, dtype=torch.int32, device="cuda"))
    table = torch.arange(-(-long // page), device="cuda").remainder(2).int().expand(9, -1).contiguous()
    q = normal(3, (n, hq, d)).cuda()
    lens = [n] * 8 + [long]
    ex.reserve_workspace(ex.attention_workspace_bytes(9, n, hq, hkv, d))
    assert not counters().any()
    got = ex.paged_attention(cache, q, ints([0, n] * 5), ints(lens), table)
    assert not counters().any()
    # the rows are the first sequence's
    want = ex.paged_attention(cache, q, ints([0] + [n] * 9), ints(lens), table)
    assert same_bits(got, want) and not counters().any()
    one = ex.paged_attention(cache, q[:1], ints([0, 1]), ints([700]), table[:1])  # split, on the same counters
    o, b = ref.attend(q[:1].cpu().double(), k[:700].cpu().double(), v[:700].cpu().double(), ref.mask(1, 700), d ** -0.5, BF16)
    ref.check(one, o, b, "after falling offsets")


def test_rows_of_no_sequence_are_not_written():
    q, k, v = normal(4, (40, 4, 64)).cuda(), normal(5, (40, 2, 64)).cuda(), normal(6, (40, 2, 64)).cuda()
    out = torch.full_like(q, 7.0)
    ex.prompt_attention(q, k, v, ints([5, 12, 3, 3, 20, 900, -4]), out=out)  # as 5, 12, 12, 12, 20, 40, 40
    want = ex.prompt_attention(q, k, v, ints([5, 12, 12, 12, 20, 40, 40]))
    assert same_bits(out[5:], want[5:]) and (out[:5] == 7.0).all()
    for a, b in ((5, 12), (12, 20), (20, 40)):
        o, e = ref.attend(*(x[a:b].cpu().double() for x in (q, k, v)), ref.mask(b - a, b - a), 0.125, BF16)
        ref.check(out[a:b], o, e, f"rows {a}..{b - 1}")


@pytest.mark.parametrize("batch", [63, 64, 65, 200])
def test_more_sequences_than_a_wave_has_lanes(batch):
    """Sequence 64 and those after it start where the 64 before them end; one offset falls."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 9, (batch,), generator=g).tolist()
    cu = torch.tensor([0] + lens).cumsum(0)
    n = int(cu[-1])
    q, k, v = normal(7, (n, 2, 64)).cuda(), normal(8, (n, 1, 64)).cuda(), normal(9, (n, 1, 64)).cuda()
    got = ex.prompt_attention(q, k, v, cu.int().cuda())
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        if b > a:
            o, e = ref.attend(*(x[a:b].cpu().double() for x in (q, k, v)), ref.mask(b - a, b - a), 0.125, BF16)
            ref.check(got[a:b], o, e, f"rows {a}..{b - 1}")
    fall = cu.clone()
    fall[40] = 1  # sequence 39 is empty, 40 begins where 39 did
    rows = slice(int(cu[39]), int(cu[41]))
    wide = ex.prompt_attention(q, k, v, fall.int().cuda())
    keep = torch.ones(n, dtype=torch.bool)
    keep[rows] = False
    assert same_bits(wide.cpu()[keep], got.cpu()[keep])
    a, b = rows.start, rows.stop
    o, e = ref.attend(*(x[a:b].cpu().double() for x in (q, k, v)), ref.mask(b - a, b - a), 0.125, BF16)
    ref.check(wide[a:b], o, e, "the sequences around the fall")


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_padding_rows_leave_the_cache_alone(bits):
    """A step of fixed size whose last rows are padding, at position -1 or of no sequence, or past the table."""
    cache = ex.KvCache.empty(6, 16, 2, 128, bits)
    every = torch.arange(96, dtype=torch.int32, device="cuda")
    x = normal(10, (96, 2, 128)).cuda()
    ex.cache_write(cache, x, x, every)
    before = ex.cache_read(cache, every)
    table = ints([[5, 1, 3], [0, 2, 4]])
    seq, pos = ints([0, 1, 1, -1, 2, 0]), ints([17, 40, -1, 3, 3, 48])
    slots = cache.slots(table, seq, pos)
    assert slots.tolist() == [17, 72, -1, -1, -1, -1]
    r = ex.Rope.make(128, 1e4, 100)
    y = normal(11, (6, 2, 128)).cuda()
    ex.rope_cache_write(cache, r, pos, slots, y, y, y)
    after = ex.cache_read(cache, every)
    keep = [i for i in range(96) if i not in (17, 72)]
    for a, b in zip(after, before):
        assert same_bits(a[keep], b[keep])
    for i, s in ((0, 17), (1, 72)):
        assert torch.equal(after[1][s].double().cpu(), ref.quantise(y[i].cpu(), bits))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,keys", [(1, 5000), (7, 9000), (200, 700), (150, 6000)])  # few rows and tiles, split and whole
def test_results_in_place_of_queries(n, keys, d):
    hq, hkv, page = 8, 2, 64
    cache = ex.KvCache.empty(-(-keys // page), page, hkv, d)
    k, v = normal(12, (keys, hkv, d)).cuda(), normal(13, (keys, hkv, d)).cuda()
    ex.cache_write(cache, k, v, torch.arange(keys, dtype=torch.int32, device="cuda"))
    table = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    qkv = normal(14, (n, (hq + 2 * hkv) * d)).cuda()
    q, kn, vn = ex.split_heads(qkv, hq, hkv, d)
    rest = qkv[:, hq * d:].clone()
    cu = ints([0, n])
    want = ex.paged_attention(cache, q, cu, ints([keys]), table)
    want2 = ex.prompt_attention(q, kn, vn, cu)
    keep = q.clone()
    assert ex.paged_attention(cache, q, cu, ints([keys]), table, out=q) is q
    assert same_bits(q, want) and same_bits(qkv[:, hq * d:], rest)
    q.copy_(keep)
    ex.prompt_attention(q, kn, vn, cu, out=q)
    assert same_bits(q, want2) and same_bits(qkv[:, hq * d:], rest)
