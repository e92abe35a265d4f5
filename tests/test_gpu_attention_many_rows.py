"""GPU: calls of more workgroups than a launch has along one dimension (2^32
threads).  Inputs are one row read for all, so that they stay small."""
import pytest
import torch

import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_cache_write_of_2_to_the_28_rows():
    tokens, heads, d = 1 << 20, 128, 256  # 8 rows a workgroup: 2^25 of them
    banner(f"cache write, {tokens} tokens of {2 * heads} heads")
    cache = ex.KvCache.empty(1, 16, heads, d)
    cache.k.zero_(), cache.v.zero_()
    row = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    where = {0: 3, 12345: 5, 131071: 6, 131072: 7, 262144: 8, tokens - 1: 11}  # workgroup 2^23 begins at token 262144
    for t, s in where.items():
        slots[t] = s
    ex.cache_write(cache, row.expand(tokens, heads, d), (-row).expand(tokens, heads, d), slots)
    for s in range(16):
        want = row.expand(1, heads, d)[0] if s in where.values() else torch.zeros(heads, d, dtype=BF16, device="cuda")
        assert torch.equal(cache.k[0, :, s], want) and torch.equal(cache.v[0, :, s], -want), f"slot {s}"


@pytest.mark.parametrize("n", [1, 3])  # with 3, the first two tokens of a sequence see no key
def test_attention_of_more_sequences_and_heads_than_a_launch_has(n):
    batch, heads, d = 16384, 1024, 64  # batch + tokens / 16 work items a head: more than 2^24 workgroups
    banner(f"attention, {batch} sequences of {n} tokens, {heads} heads")
    cache = ex.KvCache.empty(1, 16, heads, d)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(1, heads, d, generator=g).to(BF16).cuda() for _ in range(2))
    ex.cache_write(cache, k, v, ints([0]))
    q = torch.randn(1, heads, d, generator=g).to(BF16).cuda().expand(batch * n, heads, d)
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
    # one key a sequence: the last row's result is its value, those before it see none
    got = ex.paged_attention(cache, q, cu, torch.ones(batch, dtype=torch.int32, device="cuda"),
                             torch.zeros(batch, 1, dtype=torch.int32, device="cuda")).view(batch, n, heads, d)
    assert torch.equal(got[:, -1], v.expand(batch, heads, d)) and not got[:, :-1].any()
