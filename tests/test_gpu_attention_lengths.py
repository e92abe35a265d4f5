"""GPU: lengths in device memory up to the type's end.  A sequence that claims
more keys than its row of the page table can have sees what it sees with a length
that no arithmetic minds, and its neighbours what they always see.  (That no look-up leaves
the table is checked without a GPU: test_attention_ranges.py.)"""
import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner
from test_gpu_step_prefix import Shared
from test_gpu_step_sinks import BF16, Paged, same_bits

pytestmark = pytest.mark.gpu

FAR = 2 ** 30 + 2 ** 20  # a window of 2^30 does not reach the table
LENGTHS = [2 ** 31 - 2 ** 21 - 1, 2 ** 31 - 2 ** 21, 2 ** 31 - 2 ** 21 + 1, 2 ** 31 - 300, 2 ** 31 - 1]


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("bits,d", [(16, 64), (8, 128), (4, 256)])
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (100, 4), (33, 200), (2 ** 30, 4)])
def test_lengths_to_the_end_of_the_type(window, sinks, n, bits, d):
    banner(f"lengths near 2^31, window {window}, sinks {sinks}, {n} tokens, {bits} bits d={d}")
    x = Paged([n, n, n], [n + 200, 320, n + 50], 4, 2, d, BF16, bits, 16, seed=20)
    call = lambda kv: ex.paged_attention(x.cache, x.q.cuda(), x.cu.cuda(), kv, x.table.cuda(), window=window, sinks=sinks)  # noqa: E731
    want = call(ints(n + 200, FAR, n + 50))
    whole = x.run(window=window, sinks=sinks)
    if window:  # nothing but the first tokens
        k, v = (ref.quantise(t[1][:max(1, sinks)], bits) for t in (x.k, x.v))
        seen = torch.ones(n, max(1, sinks), dtype=torch.bool) if sinks else torch.zeros(n, 1, dtype=torch.bool)
        ref.check(want[n:2 * n], *ref.attend(x.q[n:2 * n].double(), k, v, seen, d ** -0.5, BF16), "first tokens")
    for kv in LENGTHS:
        got = call(ints(n + 200, kv, n + 50))
        assert same_bits(got, want), f"{kv} keys"
    for at in (slice(0, n), slice(2 * n, 3 * n)):  # (their parts may be others than in the whole call)
        assert (want[at].double() - whole[at].double()).abs().max() <= 4 * 2.0 ** -8 * whole[at].double().abs().max()


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("others", [0, 260])
def test_shared_prefixes_of_such_sequences(n, others):
    x = Shared([(96, [(n, 48), (n, 64), (n, 80)])] + [(16, [(1, 2)] * others)] * (others > 0), 4, 2, 64, BF16, 8, 16, seed=21)
    cache, q, cu, kv, table = x.args()
    more = (x.group_cu.cuda(), torch.tensor(x.shared, dtype=torch.int32).cuda())
    kv[1] = FAR
    want = ex.prefix_attention(cache, q, cu, kv, table, *more)
    plain = ex.paged_attention(cache, q, cu, kv, table)
    assert (want.double() - plain.double()).abs().max() <= 4 * 2.0 ** -8 * plain.double().abs().max()
    for m in LENGTHS:
        kv[1] = m
        assert same_bits(ex.prefix_attention(cache, q, cu, kv, table, *more), want), f"{m} keys"
    kv[:3] = 2 ** 31 - 1
    got, plain = (f(cache, q, cu, kv, table, *a) for f, a in ((ex.prefix_attention, more), (ex.paged_attention, ())))
    assert (got.double() - plain.double()).abs().max() <= 4 * 2.0 ** -8 * plain.double().abs().max()
