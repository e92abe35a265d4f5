"""GPU: the rotation with norms of the heads and with several position axes,
with and without the cache write, against the definitions in 64 bits
(step_reference.py)."""
import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
import step_reference as step
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(shape, seed, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def whole(n, top, seed):
    return torch.randint(0, top, n if isinstance(n, tuple) else (n,), generator=torch.Generator().manual_seed(seed),
                         dtype=torch.int32)


def expected(x, weight, eps, r, pos):
    """(value, bound) of x [t, h, d] on the CPU."""
    y, err = (x.double(), torch.zeros(x.shape, dtype=torch.float64)) if weight is None else step.normed(x, weight, eps)
    axes = r.axes if r.axes is not None else (0,) * (r.rotary_dim // 2)
    return step.turned(y, err, r.table.cpu(), pos, axes, r.interleaved, x.dtype)


SHAPES = [(1, 1, 1, 64, 64), (3, 5, 1, 64, 16), (67, 32, 8, 128, 128), (257, 3, 3, 128, 48), (31, 24, 4, 256, 64),
          (5, 2, 1, 256, 256)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [None, 2, 3, 4])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot", SHAPES)
def test_norm_and_rope(tokens, hq, hkv, d, rot, axes, interleaved, dtype):
    banner(f"norm rope {tokens}x({hq}+{hkv})x{d} rot={rot} axes={axes} interleaved={interleaved} {dtype}")
    r = ex.Rope.make(rot, 10000.0, 5000, interleaved)
    if axes:
        r = ex.Rope(r.table, interleaved, [int(a) for a in whole(rot // 2 - 1, axes, 9)] + [axes - 1])
    pos = whole((axes, tokens) if axes else tokens, 5000, 2)
    qkv = normal((tokens, (hq + 2 * hkv) * d), 1, dtype, 3.0)
    wq, wk = normal((d,), 3, dtype, 0.3) + 1, normal((hkv, d), 4, torch.float32, 0.3) + 1
    norm = ex.HeadNorm(wq.cuda(), wk.cuda(), 1e-5)
    q, k, _ = ex.split_heads(qkv.cuda(), hq, hkv, d)  # strided views
    qc, kc, _ = ex.split_heads(qkv, hq, hkv, d)
    for n in (norm, None) if axes else (norm,):
        q_out, k_out = ex.rope(r, pos.cuda(), q, k, norm=n)
        ref.check(q_out, *expected(qc, wq if n else None, 1e-5, r, pos), "q")
        ref.check(k_out, *expected(kc, wk if n else None, 1e-5, r, pos), "k")
        assert same_bits(ex.rope(r, pos.cuda(), q, norm=n), q_out)  # q alone
    # in place on the views
    got = ex.rope(r, pos.cuda(), q, k, q_out=q, k_out=k, norm=n)
    assert same_bits(got[0], q_out) and same_bits(got[1], k_out) and same_bits(q, q_out)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [32, 128])
def test_one_axis_has_the_plain_rotations_bits(rot, interleaved):
    plain = ex.Rope.make(rot, 1e6, 300, interleaved)
    same = ex.Rope(plain.table, interleaved, [0] * (rot // 2))
    three = ex.Rope(plain.table, interleaved, [i % 3 for i in range(rot // 2)])
    q, pos = normal((41, 6, 128), 1, F16).cuda(), whole(41, 300, 2).cuda()
    want = ex.rope(plain, pos, q)
    assert same_bits(ex.rope(same, pos[None], q), want)
    assert same_bits(ex.rope(three, pos.expand(3, 41), q), want)  # all axes the same positions, one row read thrice


def test_sections():
    blocks = ex.Rope.make(64, 1e4, 10, sections=(8, 12, 12))
    assert blocks.axes == (0,) * 8 + (1,) * 12 + (2,) * 12 and blocks.n_axes == 3
    turn = ex.Rope.make(64, 1e4, 10, sections=(16, 9, 7), in_turn=True)
    assert turn.axes[:21] == (0, 1, 2) * 7 and turn.axes[21:] == (0, 1, 0, 0, 1, 0, 0, 0, 0, 0, 0)
    assert [turn.axes.count(a) for a in range(3)] == [16, 9, 7]


def test_positions_out_of_range_are_nan_in_their_axis():
    for interleaved in (False, True):
        axes = [0, 1, 2, 1, 0, 2, 2, 0] * 2
        r = ex.Rope(ex.Rope.make(32, 1e4, 50).table, interleaved, axes)
        x = normal((3, 2, 64), 4, BF16).cuda()
        pos = torch.tensor([[1, -1, 5], [2, 50, 6], [3, 49, 2 ** 31 - 1]], dtype=torch.int32)
        y = ex.rope(r, pos.cuda(), x).cpu()
        good = ex.rope(r, pos.clamp(0, 49).cuda(), x).cpu()
        for t, bad in enumerate(({}, {0, 1}, {2})):
            for i, a in enumerate(axes):
                for at in ((2 * i, 2 * i + 1) if interleaved else (i, i + 16)):
                    assert bool(torch.isnan(y[t, :, at]).all()) == (a in bad)
                    if a not in bad:
                        assert same_bits(y[t, :, at], good[t, :, at])
            assert same_bits(y[t, :, 32:], x.cpu()[t, :, 32:])
        one = ex.rope(ex.Rope(r.table, interleaved), torch.tensor([50, 3, -7], dtype=torch.int32).cuda(), x,
                      norm=ex.HeadNorm(torch.ones(64, device="cuda")))
        assert torch.isnan(one[0::2, :, :32]).all() and torch.isfinite(one[1]).all() and torch.isfinite(one[:, :, 32:]).all()


def test_norm_of_zeros_large_values_and_what_is_not_finite():
    r = ex.Rope.make(64, 1e4, 8)
    pos = torch.arange(8, dtype=torch.int32)
    w = normal((64,), 1, torch.float32) + 2
    x = normal((8, 3, 64), 2, BF16)
    x[0] = 0
    x[1] *= 1e30       # squares past fp32
    x[2, 1] = 3e38
    x[3] *= 1e-20      # far below eps
    x[4, 0, 5] = float("nan")
    x[5, 2, 40] = float("inf")
    norm = ex.HeadNorm(w.cuda(), eps=1e-6)
    got = ex.rope(r, pos.cuda(), x.cuda(), norm=norm).cpu()
    want, bound = expected(x, w, 1e-6, r, pos)
    for t in (0, 1, 2, 3, 6, 7):
        # a row whose squares are infinite is scaled by 2^-70 first: eps is left out, which is 2^-128 of its mean
        ref.check(got[t], want[t], bound[t], f"token {t}")
    assert torch.isnan(got[4, 0]).all() and torch.isfinite(got[4, 1:]).all()
    assert torch.isfinite(got[5, :2]).all()
    bad = {40, 8}  # the pair of value 40 is 8
    for i in range(64):
        # the mean is infinite: 0 for the finite values, NaN (0 * inf) for the infinite one and its pair
        assert torch.isnan(got[5, 2, i]) if i in bad else got[5, 2, i] == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 64), (128, 32), (128, 128), (256, 64), (256, 240)])
@pytest.mark.parametrize("tokens,heads", [(3, 2), (3000, 6)])  # one and two rows a lane
def test_infinities_stay_with_their_value_and_its_pair(tokens, heads, d, rot, interleaved):
    """The mean is infinite: 0 for the finite values, NaN for an infinite one and, where it turns, for its pair."""
    r = ex.Rope.make(rot, 1e4, 8, interleaved=interleaved)
    pos = torch.arange(tokens, dtype=torch.int32) % 7 + 1
    x = normal((tokens, heads, d), 5, BF16)
    norm = ex.HeadNorm((normal((d,), 6, torch.float32) + 3).cuda(), eps=1e-6)
    half = rot // 2
    pair = lambda i: i if i >= rot else i ^ 1 if interleaved else (i + half) % rot  # noqa: E731
    bad = torch.zeros(x.shape, dtype=torch.bool)
    for t, h, places in ((0, 0, (d - 1,)), (1, 1, (rot // 2,)), (2, 0, (0, d - 2, rot - 1)), (tokens - 1, heads - 1, (rot % d, d - 4))):
        for n, i in enumerate(places):
            x[t, h, i] = float("-inf") if n else float("inf")
            bad[t, h, i] = bad[t, h, pair(i)] = True
    infinite = torch.isinf(x).any(-1, keepdim=True)
    got = ex.rope(r, pos.cuda(), x.cuda(), norm=norm).cpu()
    assert torch.equal(torch.isnan(got), bad)
    assert not got[infinite & ~bad].any() and not torch.isinf(got).any()


def test_weights_one_plus_and_copies():
    r = ex.Rope.make(128, 1e4, 40)
    pos, x = whole(40, 40, 1), normal((40, 4, 128), 2, F16)
    w = normal((128,), 3, F16, 0.1)
    dev = w.cuda()
    norm = ex.HeadNorm(dev, eps=1e-3, one_plus=True)
    want, bound = expected(x, 1 + w.double(), 1e-3, r, pos)
    f = ex.rope(r, pos.cuda(), x.cuda(), norm=norm)
    dev.zero_()  # the norm has its own copy
    assert same_bits(ex.rope(r, pos.cuda(), x.cuda(), norm=norm), f)
    ref.check(f, want, bound + 1.01 * 2.0 ** -24 * want.abs() * 2, "one plus")  # 1 + w is rounded to fp32 once


CACHES = [(b, t, d) for b in (16, 8, 4) for t in (BF16, F16) for d in (64, 128, 256)]


@pytest.mark.parametrize("bits,dtype,d", CACHES)
@pytest.mark.parametrize("axes,with_norm", [(None, True), (3, True), (3, False)])
def test_cache_write(bits, dtype, d, axes, with_norm):
    banner(f"norm rope write {bits} bits {dtype} d={d} axes={axes} norm={with_norm}")
    T, hq, hkv = 37, 6, 2
    r = ex.Rope.make(d // 2, 1e4, 100, sections=(d // 16, d // 16, d // 8) if axes else None)
    pos = whole((3, T) if axes else T, 100, 1).cuda()
    q, k, v = ex.split_heads(normal((T, (hq + 2 * hkv) * d), 2, dtype).cuda(), hq, hkv, d)
    norm = ex.HeadNorm(normal((hq, d), 3, dtype).cuda(), normal((d,), 4, dtype).cuda()) if with_norm else None
    cache = ex.KvCache.empty(5, 16, hkv, d, bits, dtype)
    slots = torch.randperm(80, generator=torch.Generator().manual_seed(5))[:T].int()
    slots[3] = -1
    slots[7] = 80
    k_out = torch.empty(T, hkv, d, dtype=dtype, device="cuda")
    got = ex.rope_cache_write(cache, r, pos, slots.cuda(), q, k, v, k_out=k_out, norm=norm)
    want_q, want_k = ex.rope(r, pos, q, k, norm=norm)
    assert same_bits(got, want_q) and same_bits(k_out, want_k)
    kr, vr = (x.cpu() for x in ex.cache_read(cache, slots.cuda()))
    here = torch.ones(T, dtype=torch.bool)
    here[3] = here[7] = False
    assert torch.equal(kr.double()[here], ref.quantise(want_k.cpu(), bits)[here])
    assert torch.equal(vr.double()[here], ref.quantise(v.cpu(), bits)[here])
    assert not kr[~here].any() and not vr[~here].any()
    # in place on the views, without k_out
    again = ex.rope_cache_write(cache, r, pos, slots.cuda(), q, k, v, q_out=q, norm=norm)
    assert again is q and same_bits(q, want_q)


def test_strided_positions_rows_and_no_tokens():
    r = ex.Rope.make(64, 1e4, 90, sections=(10, 10, 12))
    norm = ex.HeadNorm(normal((64,), 1, BF16).cuda(), normal((64,), 2, BF16).cuda())
    big = whole((3, 50), 90, 3).cuda()
    x = normal((4, 20, 64), 4, BF16).cuda()  # [heads, tokens, d]
    out = torch.empty(4, 20, 64, dtype=BF16, device="cuda")
    got = ex.rope(r, big[:, 7:27], x.transpose(0, 1), q_out=out.transpose(0, 1), norm=norm)
    want = ex.rope(r, big[:, 7:27].contiguous(), x.transpose(0, 1).contiguous(), norm=norm)
    assert same_bits(got, want) and same_bits(out, want.transpose(0, 1))
    empty = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    assert ex.rope(r, big[:, :0], empty, norm=norm).shape == (0, 4, 64)
    cache = ex.KvCache.empty(1, 16, 4, 64, 8)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ex.rope_cache_write(cache, r, big[:, :0], none, empty, empty, empty, norm=norm).shape == (0, 4, 64)


def test_rows_past_32_bit_offsets():
    """Rows more than 2^32 values apart."""
    r = ex.Rope.make(64, 1e4, 90)
    norm = ex.HeadNorm(normal((64,), 1, BF16).cuda())
    far = torch.zeros(2 ** 32 + 4096, dtype=BF16, device="cuda")
    x = normal((2, 3, 64), 2, BF16)
    q = far.as_strided((2, 3, 64), (2 ** 32 + 64, 128, 1))
    q.copy_(x)
    pos = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    got = ex.rope(r, pos, q, q_out=q, norm=norm)
    assert same_bits(got, ex.rope(r, pos, x.cuda(), norm=norm))


def test_on_another_stream_and_in_a_graph():
    r = ex.Rope.make(128, 1e4, 90, sections=(20, 22, 22))
    norm = ex.HeadNorm(normal((128,), 1, BF16).cuda(), normal((128,), 2, BF16).cuda())
    q, k, v = (normal((9, h, 128), h, BF16).cuda() for h in (8, 2, 2))
    pos, slots = whole((3, 9), 90, 3).cuda(), torch.arange(9, dtype=torch.int32, device="cuda")
    cache = ex.KvCache.empty(2, 16, 2, 128, 8)
    want = ex.rope_cache_write(cache, r, pos, slots, q, k, v, norm=norm)
    want_k = ex.cache_read(cache, slots)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ex.rope_cache_write(cache, r, pos, slots, q, k, v, q_out=out, norm=norm)
    for i in range(3):
        out.zero_()
        cache.k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want) and same_bits(ex.cache_read(cache, slots)[0], want_k), f"replay {i}"
