"""GPU: float16 attention where most keys have weights below the type's normal
range.

Every 32nd key has score 0 and the value 0, the others a score of about
ln(1.5 * 2^-24) and the value 1024, so the exact result is
1024 * 31 w / (1 + 31 w) with w near 9e-8.  A probability is rounded to the type
with the row's maximum at 2^7 at least, so what its rounding adds to the
relative 2^-11 is at most 2^-25 a key (half the spacing of subnormals), against
a sum of at least 2^7 for every 32 keys: 31 * 1024 * 2^-32 = 7.4e-6 of a result
of 2.8e-3.  With the maximum at 1 it would be a third of the result."""
import math

import pytest
import torch

import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def inputs(n, keys, d, score):
    k = torch.zeros(keys, 1, d, dtype=torch.float16)
    k[:, 0, 0] = score
    k[::32, 0, 0] = 0
    v = torch.full((keys, 1, d), 1024, dtype=torch.float16)
    v[::32] = 0
    q = torch.zeros(n, 1, d, dtype=torch.float16)
    q[:, 0, 0] = 1
    return q.cuda(), k.cuda(), v.cuda()


def check(got, seen, score):
    """seen: the keys that each row sees."""
    few = (seen + 31) // 32
    w = math.exp(score)
    want = ((seen - few) * 1024 * w / (few + (seen - few) * w))[:, None]
    rounding = 31 * 1024 * 2.0 ** -32
    err = 1.01 * (U + 2.0 ** -23 * 200) * want + rounding  # scores are exact; a few roundings of exp2 and the sums
    bound = U * (want + err) + err + 2.0 ** -25
    diff = (got.double().cpu()[:, 0] - want).abs()
    assert (diff <= bound).all(), f"worst {float((diff - bound).max()):.3e} over, of {float(want.max()):.3e}"


@pytest.mark.parametrize("score", [-16.234375, -16.21875])  # 1.494 and 1.518 times 2^-24
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 200])
def test_cached_keys(n, d, score):
    banner(f"small weights, cached, n={n} d={d} {score}")
    keys, page = 6400, 64
    q, k, v = inputs(n, keys, d, score)
    cache = ex.KvCache.empty(keys // page, page, 1, d, 16, torch.float16)
    ex.cache_write(cache, k, v, torch.arange(keys, dtype=torch.int32, device="cuda"))
    got = ex.paged_attention(cache, q, torch.tensor([0, n], dtype=torch.int32).cuda(),
                             torch.tensor([keys], dtype=torch.int32).cuda(),
                             torch.arange(keys // page, dtype=torch.int32, device="cuda")[None], scale=1.0)
    check(got, torch.arange(keys - n + 1, keys + 1).double(), score)


@pytest.mark.parametrize("score", [-16.234375, -16.21875])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [40, 2048])
def test_prompts(n, d, score):
    banner(f"small weights, prompt, n={n} d={d} {score}")
    q, k, v = inputs(n, n, d, score)
    got = ex.prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32).cuda(), scale=1.0)
    check(got, torch.arange(1, n + 1).double(), score)
