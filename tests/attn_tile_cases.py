"""Calls that the GPU tests make to reach the attention kernel for many rows, and
whether their keys are split; the host's choice of both is checked without a
GPU.  Not collected by pytest."""


def call(name, q_lens, kv_lens, hq, hkv, d, split, prompt=False):
    return dict(name=name, q_lens=q_lens, kv_lens=kv_lens, hq=hq, hkv=hkv, d=d, split=split, prompt=prompt)


# chunks over every format of heads of 256, beside a sequence without new tokens (the plan splits, the keys are too few)
CHUNKS = call("chunks", [70, 0, 150], [200, 40, 333], 6, 2, 256, True)
# a chunk in a cache of more than 4 GB
FAR = call("far pages", [150], [300], 8, 8, 256, True)
# a chunk over enough keys that each tile has ten parts (of 1024 keys at least), two levels of their tree
LONG = {d: call(f"long chunk, heads of {d}", [70], [10100], 2, 1, d, True) for d in (64, 128, 256)}
# prompts whose tiles have several parts
PROMPTS = {d: call(f"long prompt, heads of {d}", [2600, 130], [2600, 130], 2, 1, d, True, True) for d in (64, 128, 256)}
# enough tiles that nothing is split
FULL = {d: call(f"many tiles, heads of {d}", [700] * 4, [1500, 700, 800, 9000], 128, 32, d, False) for d in (64, 128, 256)}

ALL = [CHUNKS, FAR, *LONG.values(), *PROMPTS.values(), *FULL.values()]
