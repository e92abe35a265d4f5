"""GPU: bfloat16 attention over values near the type's largest.

A result is an average of values, so it is in range wherever they are.  The sums
of probability times value must not overflow on the way, neither where a running
maximum lags behind scores that rise by steps nor where a wave or a part of the
keys has only such as weigh nothing in the end."""
import math

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("step", [2.0, 5.25, 7.5])  # in powers of two
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 6, 300])  # few rows, few rows of one sequence, tiles
def test_values_near_the_largest(n, d, step):
    banner(f"large values n={n} d={d} step={step}")
    keys = 13 * 128
    q = torch.zeros(n, 2, d).to(BF16)
    q[:, :, 0] = 1
    k = torch.zeros(keys, 1, d).to(BF16)
    # of every 128 keys (which no wave or tile reads past in one step) one weighs 2^step times that of those before, and
    # the others nothing
    rise = torch.tensor([i // 128 * step - (0 if i % 128 == 5 else 60.0) for i in range(keys)]) * math.log(2)
    k[:, 0, 0] = rise.to(BF16)
    v = torch.full((keys, 1, d), 2.0 ** 126).to(BF16)
    v[:, :, 1::2] = -(2.0 ** 126)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cache = ex.KvCache.empty(-(-keys // 64), 64, 1, d)
    ex.cache_write(cache, k.cuda(), v.cuda(), torch.arange(keys, dtype=torch.int32, device="cuda"))
    got = ex.paged_attention(cache, q.cuda(), cu, torch.tensor([keys], dtype=torch.int32, device="cuda"),
                             torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None], scale=1.0)
    # the definition on scaled values, exact by powers of two
    o, b = ref.attend(q.double(), k.double(), v.double() * 2.0 ** -126, ref.mask(n, keys), 1.0, BF16)
    ref.check(got.double().cpu() * 2.0 ** -126, o, b, "cached")
    got = ex.prompt_attention(q.cuda(), k[:n].cuda(), v[:n].cuda(), cu, scale=1.0)
    o, b = ref.attend(q.double(), k[:n].double(), v[:n].double() * 2.0 ** -126, ref.mask(n, n), 1.0, BF16)
    ref.check(got.double().cpu() * 2.0 ** -126, o, b, "prompt")
