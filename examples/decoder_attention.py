"""The attention half of a decoder layer, from the layer's input to the output
projection, with EXL3 weights and a paged cache: prompts first, then one new
token at a time.

    python examples/decoder_attention.py [--bits 8] [--steps 32]

Random weights of a layer with a 4096 model dimension, 32 query and 8
key/value heads of 128.  The step's sizes are fixed and nothing reads the GPU
back, so it is captured once as a graph and replayed.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_exl3_input_amd as ex  # noqa: E402


def random_weight(K, shards, bits, codebook="mul1", seed=0):
    """An EXL3 weight whose trellis is uniformly random, scaled to about unit gain."""
    g = torch.Generator("cuda").manual_seed(seed)
    N = sum(shards)
    trellis = torch.randint(-32768, 32768, (K // 16, N // 16, 16 * bits), generator=g, device="cuda",
                            dtype=torch.int32).to(torch.int16)

    def signs(*shape):
        return torch.randint(0, 2, shape, generator=g, device="cuda").mul(2).sub(1).half()

    return ex.Exl3Weight(trellis, signs(len(shards), K), signs(N) * K ** -0.5, bits, codebook, shards)


class AttentionBlock:
    """q/k/v projection, rotary positions, cache, attention and output projection of one layer."""

    def __init__(self, w_qkv, w_o, rope, cache, q_heads):
        self.w_qkv, self.w_o, self.rope, self.cache = w_qkv, w_o, rope, cache
        self.q_heads, self.kv_heads, self.head_dim = q_heads, cache.heads, cache.head_dim

    def project(self, x, positions, slots):
        """q rotated, and k rotated and v as they are kept; the cache holds k and v afterwards."""
        qkv = ex.forward(self.w_qkv, x)
        q, k, v = ex.split_heads(qkv, self.q_heads, self.kv_heads, self.head_dim)
        ex.rope_cache_write(self.cache, self.rope, positions, slots, q, k, v, q_out=q, k_out=k)  # in place
        return q, k, v

    def output(self, y):
        return ex.forward(self.w_o, y.view(y.shape[0], -1))

    def prompt(self, x, cu, positions, slots):
        """Whole prompts packed one after another: attention over the tokens' own keys and values."""
        q, k, v = self.project(x, positions, slots)
        return self.output(ex.prompt_attention(q, k, v, cu))

    def extend(self, x, cu, kv_len, page_table, positions, slots):
        """New tokens (one, a few drafted, or a chunk of a prompt) of sequences that are in the cache."""
        q, _, _ = self.project(x, positions, slots)
        return self.output(ex.paged_attention(self.cache, q, cu, kv_len, page_table))


def pages_of(capacity, page_size):
    """A page table for sequences of at most `capacity` tokens each, and the pages it needs."""
    each = [-(-n // page_size) for n in capacity]
    table = torch.full((len(each), max(each)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(each)).int(), 0
    for s, n in enumerate(each):
        table[s, :n] = order[at:at + n]
        at += n
    return table.cuda(), sum(each)


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--bits", type=int, default=8, choices=(16, 8, 4), help="bits of the cache")
    a.add_argument("--steps", type=int, default=32)
    a.add_argument("--page", type=int, default=64)
    a = a.parse_args()
    dim, hq, hkv, d = 4096, 32, 8, 128
    lens = [1500, 4000, 17, 800]
    table, pages = pages_of([n + a.steps for n in lens], a.page)
    block = AttentionBlock(random_weight(dim, (hq * d, hkv * d, hkv * d), 4, seed=1), random_weight(hq * d, (dim,), 4, seed=2),
                           ex.Rope.make(d, 1e6, 32768), ex.KvCache.empty(pages, a.page, hkv, d, a.bits), hq)

    # ---- the prompts
    B, T = len(lens), sum(lens)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(lens, device="cuda"))
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    slots = block.cache.slots(table, seq, positions)
    x = torch.randn(T, dim, device="cuda").bfloat16()
    for name in ("first call", "again"):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y = block.prompt(x, cu, positions, slots)
        torch.cuda.synchronize()
        print(f"{B} prompts, {T} tokens: {(time.perf_counter() - t0) * 1e6:.0f} us ({name}), finite {bool(y.isfinite().all())}")

    # ---- one token a sequence and step: captured once, replayed
    cu1 = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    every = torch.arange(B, device="cuda")
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")  # before the step's own token
    x1 = x[:B].clone()

    def step():
        pos = kv_len.clone()
        kv_len.add_(1)
        return block.extend(x1, cu1, kv_len, table, pos, block.cache.slots(table, every, pos))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        kv_len.sub_(1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y1 = step()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            graph.replay()
            x1.copy_(y1.clamp(-4, 4))  # the next step's input
        torch.cuda.synchronize()
    print(f"{a.steps} steps of {B} sequences: {(time.perf_counter() - t0) / a.steps * 1e6:.0f} us each, "
          f"lengths {kv_len.tolist()}, finite {bool(y1.isfinite().all())}")


if __name__ == "__main__":
    main()
