"""GPU: the attention half of a decoder layer as examples/decoder_attention.py
runs it, from the layer's input to the output projection.

Prompts, chunks and single tokens have to agree: each attention output is
within 2 roundings of the exact one (the probabilities' and the output's, each
at most 2^-9 of the largest |v| for bfloat16), so two of them within 4, and
1/16 of that is left for the fp32 sums."""
import importlib.util
import os

import pytest
import torch

import linear_exl3_input_amd as ex
from gpu_util import banner

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def demo():
    ex.load()
    spec = importlib.util.spec_from_file_location("decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def weights(demo):
    return demo.random_weight(512, (512, 256, 256), 4, seed=1), demo.random_weight(512, (512,), 4, seed=2)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_prompts_chunks_and_steps_agree(demo, weights, bits):
    banner(f"decoder attention, {bits}-bit cache")
    torch.manual_seed(bits)
    lens, page = [70, 1, 33], 16
    table, pages = demo.pages_of(lens, page)
    block = demo.AttentionBlock(*weights, ex.Rope.make(64, 1e4, 128), ex.KvCache.empty(pages, page, 2, 128, bits), 4)
    x = [torch.randn(n, 512, device="cuda").bfloat16() for n in lens]

    # prompts whole
    cu = ints([0, 70, 71, 104])
    seq = torch.repeat_interleave(torch.arange(3, device="cuda"), cu.diff().long())
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
    slots = block.cache.slots(table, seq, pos)
    q, k, v = block.project(torch.cat(x), pos, slots)
    whole = ex.prompt_attention(q, k, v, cu)
    assert torch.equal(block.output(whole), block.prompt(torch.cat(x), cu, pos, slots))
    # what the cache holds instead of k and v
    kc, vc = ex.cache_read(block.cache, slots)
    if bits == 16:
        assert torch.equal(kc, k.contiguous()) and torch.equal(vc, v.contiguous())
    cached = ex.prompt_attention(q, kc, vc, cu)

    # the same tokens into an empty cache: chunks of different sizes, then one by one
    cache2 = ex.KvCache.empty(pages, page, 2, 128, bits)
    block2 = demo.AttentionBlock(*weights, block.rope, cache2, 4)
    got = torch.zeros_like(cached)
    done = [0, 0, 0]
    for sizes in ([40, 0, 17], [5, 1, 15], *[[1, 0, int(i == 0)] for i in range(25)]):
        tok = [torch.arange(d, d + n, device="cuda") for d, n in zip(done, sizes)]
        at = torch.cat([t + int(c) for t, c in zip(tok, cu.tolist())])
        p = torch.cat(tok).int()
        s = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sizes, device="cuda"))
        done = [d + n for d, n in zip(done, sizes)]
        q2, _, _ = block2.project(torch.cat(x)[at], p, cache2.slots(table, s, p))
        assert torch.equal(q2, q[at])
        got[at] = ex.paged_attention(cache2, q2, ints([0, *torch.tensor(sizes).cumsum(0).tolist()]), ints(done), table)
    assert done == lens
    for a, b in zip(ex.cache_read(cache2, slots), (kc, vc)):
        assert torch.equal(a, b)
    for s in range(3):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        bound = 4 * 2.0 ** -9 * vc[rows].abs().max().item() * (1 + 1 / 16)
        err = (got[rows].float() - cached[rows].float()).abs().max().item()
        assert err <= bound, f"sequence {s}: {err} over {bound}"
