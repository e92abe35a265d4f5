"""GPU: rotary positions and the cache's write and read, against their
definitions in 64 bits (attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(shape, seed, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot", [(1, 1, 1, 64, 64), (3, 5, 1, 64, 16), (67, 32, 8, 128, 128),
                                                 (257, 3, 3, 128, 48), (31, 24, 4, 256, 64), (5, 2, 1, 256, 256)])
def test_rope(tokens, hq, hkv, d, rot, interleaved, dtype):
    banner(f"rope {tokens}x({hq}+{hkv})x{d} rot={rot} interleaved={interleaved} {dtype}")
    r = ex.Rope.make(rot, 10000.0, 5000, interleaved, yarn=(4.0, 1000))
    qkv = normal((tokens, (hq + 2 * hkv) * d), 1, dtype)
    pos = torch.randint(0, 5000, (tokens,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    q, k, _ = ex.split_heads(qkv.cuda(), hq, hkv, d)  # strided views
    q_out, k_out = ex.rope(r, pos.cuda(), q, k)
    table = r.table.cpu()
    qc, kc, _ = ex.split_heads(qkv, hq, hkv, d)
    ref.check(q_out, *ref.rotate(qc, table, pos, interleaved), "q")
    ref.check(k_out, *ref.rotate(kc, table, pos, interleaved), "k")
    # q alone, and in place on the views
    assert same_bits(ex.rope(r, pos.cuda(), q), q_out)
    got = ex.rope(r, pos.cuda(), q, k, q_out=q, k_out=k)
    assert same_bits(got[0], q_out) and same_bits(got[1], k_out) and same_bits(q, q_out)


def test_rope_head_major_and_shared_rows():
    r = ex.Rope.make(64, 10000.0, 100)
    x = normal((4, 7, 64), 3, BF16)  # [heads, tokens, d]
    pos = torch.arange(7, dtype=torch.int32)
    want = ex.rope(r, pos.cuda(), x.transpose(0, 1).contiguous().cuda())
    out = torch.empty(4, 7, 64, dtype=BF16, device="cuda")
    got = ex.rope(r, pos.cuda(), x.cuda().transpose(0, 1), q_out=out.transpose(0, 1))
    assert same_bits(got, want) and same_bits(out, want.transpose(0, 1))
    one = x[:1].cuda().expand(4, 7, 64).transpose(0, 1)  # one head read as four
    got = ex.rope(r, pos.cuda(), one)
    assert all(same_bits(got[:, h], want[:, 0]) for h in range(4))


def test_rope_position_out_of_range_is_nan():
    r = ex.Rope.make(32, 10000.0, 50)
    x = normal((4, 2, 64), 4, F16).cuda()
    y = ex.rope(r, torch.tensor([-1, 49, 50, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), x)
    for t, bad in enumerate((True, False, True, True)):
        assert bool(torch.isnan(y[t, :, :32]).all()) == bad
        assert same_bits(y[t, :, 32:], x[t, :, 32:])


def test_rope_no_tokens():
    r = ex.Rope.make(64, 10000.0, 4)
    empty = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    assert ex.rope(r, torch.empty(0, dtype=torch.int32, device="cuda"), empty).shape == (0, 2, 64)


def test_rope_tables():
    plain = ex.Rope.make(64, 10000.0, 300).table.double().cpu()
    inv = 10000.0 ** -(torch.arange(32).double() / 32)
    a = torch.arange(300).double()[:, None] * inv
    assert (plain - torch.stack((a.cos(), a.sin()), -1)).abs().max() <= 2.0 ** -24
    linear = ex.Rope.make(64, 10000.0, 300, linear=2.0).table.cpu()
    assert (linear[::2].double() - plain[:150]).abs().max() <= 2.0 ** -23
    # ntk: the fastest pair stays, the slowest slows by the factor
    ntk = ex.Rope.make(64, 10000.0, 300, ntk=4.0).table.double().cpu()
    assert (ntk[:, 0] - plain[:, 0]).abs().max() == 0
    assert math.isclose(math.atan2(ntk[299, 31, 1], ntk[299, 31, 0]), 299 * inv[31].item() / 4, rel_tol=1e-4)
    yarn = ex.Rope.make(64, 10000.0, 300, yarn=(4.0, 100), yarn_gain=1.0).table.double().cpu()
    turns = 100 * inv / (2 * math.pi)
    slow = turns < 1
    b = torch.arange(300).double()[:, None] * torch.where(slow, inv / 4, inv)
    keep = slow | (turns > 32)
    assert (yarn - torch.stack((b.cos(), b.sin()), -1))[:, keep].abs().max() <= 2.0 ** -24
    gain = ex.Rope.make(64, 10000.0, 300, yarn=(4.0, 100)).table.double().cpu()
    assert (gain - yarn * (0.1 * math.log(4.0) + 1)).abs().max() <= 2.0 ** -22


CACHES = [(b, t, d) for b in (16, 8, 4) for t in (BF16, F16) for d in (64, 128, 256)]


@pytest.mark.parametrize("bits,dtype,d", CACHES)
@pytest.mark.parametrize("heads,page,tokens", [(1, 16, 1), (3, 16, 37), (8, 256, 300)])
def test_cache_write_and_read(bits, dtype, d, heads, page, tokens):
    banner(f"cache {bits} bits {dtype} d={d} heads={heads} page={page} tokens={tokens}")
    pages = -(-tokens // page) + 2
    cache = ex.KvCache.empty(pages, page, heads, d, bits, dtype)
    k = normal((tokens, heads, d), 5, dtype, torch.exp2(3 * torch.randn(heads, d, generator=torch.Generator().manual_seed(6))))
    v = normal((tokens, heads, d), 7, dtype)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(8))[:tokens].int()
    ex.cache_write(cache, k.cuda(), v.cuda(), slots.cuda())
    kr, vr = ex.cache_read(cache, slots.cuda())
    assert kr.dtype == dtype and kr.shape == (tokens, heads, d)
    for got, x in ((kr, k), (vr, v)):
        want = ref.quantise(x, bits)
        assert torch.equal(want.to(dtype).double(), want)  # exact in the type
        assert torch.equal(got.cpu().double(), want)


def special_blocks(dtype):
    """One head of 256 values: eight blocks with what quantizing can trip over."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    b = torch.zeros(8, 32)
    b[0, 3] = math.nan
    b[1, 7], b[1, 8] = math.inf, 1.0
    b[2, 31] = -math.inf
    # b[3]: zeros, one of them negative
    b[3, 0] = -0.0
    b[4] = torch.linspace(-big, big, 32)
    b[5] = torch.linspace(-1, 1, 32) * tiny / 4
    b[6] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 7.0] * 2)
    b[7] = torch.tensor([1.0625, 1.1875, 448.0, -440.0, 432.0, 2.0 ** -9, 3 * 2.0 ** -10, 2.0 ** -10] * 4)
    return b.reshape(256).to(dtype)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cache_special_values(bits, dtype):
    x = special_blocks(dtype).reshape(1, 1, 256)
    cache = ex.KvCache.empty(2, 16, 1, 256, bits, dtype)
    slots = torch.tensor([17], dtype=torch.int32, device="cuda")
    ex.cache_write(cache, x.cuda(), (-x).cuda(), slots)
    k, v = ex.cache_read(cache, slots)
    for got, src in ((k, x), (v, -x)):
        want = ref.quantise(src, bits)
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(got.cpu().double().nan_to_num(0.0, 7.0, -7.0), want.nan_to_num(0.0, 7.0, -7.0))


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_cache_skips_slots_out_of_range(bits):
    cache = ex.KvCache.empty(3, 16, 2, 128, bits, BF16)
    every = torch.arange(48, dtype=torch.int32, device="cuda")
    base = normal((48, 2, 128), 9, BF16).cuda()
    ex.cache_write(cache, base, base, every)
    before = ex.cache_read(cache, every)
    k = normal((5, 2, 128), 10, BF16).cuda()
    slots = torch.tensor([-1, 5, 48, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    ex.cache_write(cache, k, k, slots)
    after = ex.cache_read(cache, every)
    rest = [i for i in range(48) if i != 5]
    assert same_bits(after[0][rest], before[0][rest]) and same_bits(after[1][rest], before[1][rest])
    assert torch.equal(after[0][5].cpu().double(), ref.quantise(k[1].cpu(), bits))
    back = ex.cache_read(cache, slots)
    assert torch.equal(back[0][[0, 2, 3, 4]], torch.zeros(4, 2, 128, dtype=BF16, device="cuda"))
    assert same_bits(back[0][1], after[0][5])


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("dtype,interleaved", [(BF16, False), (F16, True)])
def test_fused_write_has_the_bits_of_the_two_calls(bits, dtype, interleaved):
    T, hq, hkv, d = 41, 12, 3, 128
    r = ex.Rope.make(96, 10000.0, 2000, interleaved)
    qkv = normal((T, (hq + 2 * hkv) * d), 11, dtype).cuda()
    q, k, v = ex.split_heads(qkv, hq, hkv, d)
    g = torch.Generator().manual_seed(12)
    pos = torch.randint(0, 2000, (T,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(96, generator=g)[:T].int().cuda()
    slots[3] = -1
    a, b = (ex.KvCache.empty(6, 16, hkv, d, bits, dtype) for _ in range(2))
    q1, k1 = ex.rope(r, pos, q, k)
    ex.cache_write(a, k1, v, slots)
    k2 = torch.empty_like(k1)
    q2 = ex.rope_cache_write(b, r, pos, slots, q, k, v, k_out=k2)
    assert same_bits(q1, q2) and same_bits(k1, k2)
    for x, y in zip(ex.cache_read(a, slots), ex.cache_read(b, slots)):
        assert same_bits(x, y)
    # in place on the projection's output, nothing else of it touched
    v0 = v.clone()
    ex.rope_cache_write(b, r, pos, slots, q, k, v, q_out=q, k_out=k)
    assert same_bits(q, q1) and same_bits(k, k1) and same_bits(v, v0)


def test_cache_of_one_layer_in_a_tensor_for_all():
    layers = torch.zeros(5, 3, 2, 16, 128, dtype=torch.uint8, device="cuda")  # [pages, layers, heads, page, d]
    scales = torch.zeros(5, 3, 2, 16, 4, dtype=torch.uint8, device="cuda")
    caches = [ex.KvCache(layers[:, i], layers.clone()[:, i], scales[:, i], scales.clone()[:, i], BF16) for i in range(3)]
    x = normal((80, 2, 128), 13, BF16)
    slots = torch.arange(80, dtype=torch.int32, device="cuda")
    ex.cache_write(caches[1], x.cuda(), x.cuda(), slots)
    k, v = ex.cache_read(caches[1], slots)
    assert torch.equal(k.cpu().double(), ref.quantise(x, 8)) and same_bits(k, v)
    assert not layers[:, 0].any() and not layers[:, 2].any() and not scales[:, 0].any() and not scales[:, 2].any()


def test_cache_past_four_gigabytes():
    pages, page, heads, d = 5200, 256, 8, 256  # 5.4 GB of keys at 16 bits
    cache = ex.KvCache.empty(pages, page, heads, d, 16, BF16)
    x = normal((3, heads, d), 14, BF16).cuda()
    slots = torch.tensor([pages * page - 1, 0, 4100 * page + 7], dtype=torch.int32, device="cuda")
    cache.k[0, :, 0] = 0
    ex.cache_write(cache, x, -x, slots)
    k, v = ex.cache_read(cache, slots)
    assert same_bits(k, x) and same_bits(v, -x)
    assert same_bits(cache.k[pages - 1, :, page - 1], x[0]) and same_bits(cache.k[4100, :, 7], x[2])


def test_slots_of_positions():
    cache = ex.KvCache.empty(10, 16, 1, 64, 16, BF16)
    table = torch.tensor([[4, 2, -1], [7, 9, 0]], dtype=torch.int32, device="cuda")
    got = cache.slots(table, torch.tensor([0, 0, 0, 1, 1], device="cuda"), torch.tensor([0, 17, 40, 31, 32], device="cuda"))
    assert got.tolist() == [64, 33, -1, 159, 0] and got.dtype == torch.int32


def test_rotations_on_another_device_are_refused():
    r = ex.Rope.make(64, 1e4, 32)
    x = torch.randn(2, 4, 64, device="cuda").bfloat16()
    cache = ex.KvCache.empty(1, 16, 4, 64)
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    r.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="the rotations are on cuda:1, q on cuda:0"):
        ex.rope(r, at, x)
    with pytest.raises(ValueError, match="the rotations are on cuda:1, q on cuda:0"):
        ex.rope_cache_write(cache, r, at, at, x, x, x)
