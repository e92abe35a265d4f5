"""The work of a serving step's operators: block tables and slot maps from
request lengths, norms of query and key heads with the rotation (of one or of
several position axes) in the same pass, attention with a window and first
tokens that stay visible, and attention of a batch whose sequences share a
prefix.

``listed()`` names the measured cases and ``draw()`` gives more of the same
ranges.  ``prepare`` makes a case's inputs, ``run`` one pass: with ``own``
false the plain form (elementary torch operations in 32 bits, rounded once at
the end), with ``own`` true this package's calls.  ``exact`` is the same
definition in 64 bits, one sequence at a time.

The cache's format: 16 bits hold the values; 8 and 4 bits hold blocks of 32
values along the head as e4m3 or e2m1 codes (4 bits: two in a byte, the even
index in the low half) and a byte s per block, the value being
code * 2^(s - 127).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F16 = "bf16", "fp16"
DTYPES = {BF16: torch.bfloat16, F16: torch.float16}
EPS = 1e-6

# The least and greatest exponent of a block's scale: every stored value is
# then exact in the cache's 16-bit type.
SCALE_RANGE = {(BF16, 8): (-117, 119), (BF16, 4): (-125, 125), (F16, 8): (-15, 7), (F16, 4): (-23, 13)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of 64 requests: a token each, and now and then a page.
        dict(name="tables_step", op="tables", batch=64, q_max=1, kv_max=9000, page=64),
        # A step that admits many prompts and continues others: most pages are new.
        dict(name="tables_prompts", op="tables", batch=300, q_max=1500, kv_max=4000, page=16),
        # One step of 16 sequences, heads of 256 of which a quarter turns, normed and rotated.
        dict(name="norm_step", op="rows", tokens=16, hq=24, hkv=4, d=256, rot=64, interleaved=False, dtype=BF16,
             norm=True, axes=1, cycle=False, bits=0, page=64),
        # A long prompt normed, rotated and written to an 8-bit cache, then read back.
        dict(name="norm_write_prompt", op="rows", tokens=12001, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype=BF16, norm=True, axes=1, cycle=False, bits=8, page=64),
        # A video's tokens: time, height and width turn their own pairs, in blocks.
        dict(name="axes_video", op="rows", tokens=9973, hq=32, hkv=8, d=128, rot=128, interleaved=False, dtype=F16,
             norm=False, axes=3, cycle=False, bits=0, page=64),
        # A step of 48 sequences: three axes in turn, written to a 4-bit cache in the same call and read back.
        dict(name="axes_write_step", op="rows", tokens=48, hq=32, hkv=8, d=128, rot=128, interleaved=True, dtype=BF16,
             norm=False, axes=3, cycle=True, bits=4, page=64),
        # Endless generation: one token of 32 sequences, pages between the first tokens and the window given back.
        dict(name="sinks_step", op="paged", batch=32, q_max=1, kv_max=40000, hq=32, hkv=8, d=128, dtype=BF16, bits=8,
             page=64, window=4096, sinks=4, freed=True),
        # Chunks of long prompts.
        dict(name="sinks_chunk", op="paged", batch=3, q_max=900, kv_max=15000, hq=32, hkv=8, d=128, dtype=F16, bits=16,
             page=32, window=2048, sinks=100, freed=False),
        # Whole prompts packed together, wide heads.
        dict(name="sinks_prompt", op="prompt", batch=3, len_max=6000, hq=24, hkv=4, d=256, dtype=BF16, window=1024,
             sinks=16),
        # A few answers to one question of moderate length.
        dict(name="prefix_few", op="prefix", batch=4, groups=1, q_max=1, prefix=960, own_max=150, hq=32, hkv=8, d=128,
             dtype=BF16, bits=16, page=64),
        # A busy server whose requests start with the same long instructions.
        dict(name="prefix_batch", op="prefix", batch=64, groups=1, q_max=1, prefix=24000, own_max=1500, hq=32, hkv=8,
             d=128, dtype=BF16, bits=8, page=64),
        # Several documents, each with its own questions of some tokens, narrow heads.
        dict(name="prefix_questions", op="prefix", batch=40, groups=3, q_max=24, prefix=9000, own_max=600, hq=16, hkv=4,
             d=64, dtype=F16, bits=16, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "rows", "rows", "paged", "prompt", "prefix", "prefix"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "tables":
        batch = _log(rng, 1, 400)
        return dict(op=op, batch=batch, q_max=rng.choice((1, 1, _log(rng, 2, min(2000, 150000 // batch)))), kv_max=_log(rng, 16, 10000),
                    page=page)
    d = rng.choice((64, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 6, 8))
    case = dict(op=op, hq=hq, hkv=hkv, d=d, dtype=rng.choice((BF16, F16)))
    if op == "rows":
        axes = rng.choice((1, 2, 3, 3))
        norm = axes == 1 or rng.random() < 0.5
        case.update(tokens=_log(rng, 1, 7000 * 4096 // max(4096, hq * d)), rot=rng.choice((d // 4, d // 2, d)), interleaved=rng.random() < 0.5,
                    norm=norm, axes=axes, cycle=rng.random() < 0.5, bits=rng.choice((0, 16, 8) if norm else (0, 8, 4)),
                    page=page)
    if op == "paged":
        q = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 700)))
        batch = _log(rng, 1, 32 if q <= 16 else 4)
        kv = max(q, _log(rng, 16, 30000 if batch <= 8 and q <= 16 else 10000))
        window = _log(rng, 30, 4096)
        case.update(bits=rng.choice((16, 8, 4)), page=page, batch=batch, q_max=q, kv_max=kv, window=window,
                    sinks=rng.choice((1, 4, _log(rng, 2, 300))), freed=rng.random() < 0.5)
    if op == "prompt":
        batch = _log(rng, 1, 24)
        case.update(hq=min(hq, 8192 // d), batch=batch, len_max=_log(rng, 2, 4000 // max(1, batch - 1)),
                    window=_log(rng, 30, 1300), sinks=rng.choice((1, 4, _log(rng, 2, 200))))
    if op == "prefix":
        q = rng.choice((1, 1, 1, _log(rng, 2, 40)))
        batch = _log(rng, 2, 48 if q == 1 else 16)
        case.update(bits=rng.choice((16, 8, 4)), page=page, batch=batch, groups=rng.randint(1, min(4, batch)), q_max=q,
                    prefix=_log(rng, 200, 12000 if q == 1 else 5000), own_max=max(q, _log(rng, 1, 1500)))
    return case


def _lengths(case):
    """New tokens and keys of a case's sequences: the first as long as
    stated, the others spread from very short to that, the same for every
    seed."""
    r = np.random.RandomState(1234 + case["batch"])
    spread = lambda top: [top] + [max(1, int(top * r.uniform(0.02, 1.0) ** 1.5)) for _ in range(case["batch"] - 1)]  # noqa: E731
    if case["op"] == "prompt":
        lens = spread(case["len_max"])
        return lens, lens
    if case["op"] == "tables":
        # requests that wait are in the batch without a token, new ones without a past
        q = [1] * case["batch"] if case["q_max"] == 1 else spread(case["q_max"])
        kv = [0 if r.randint(8) == 0 else n - 1 for n in spread(case["kv_max"])]
        return [0 if i and r.randint(10) == 0 else n for i, n in enumerate(q)], kv
    lens = spread(case["own_max"] if case["op"] == "prefix" else case["kv_max"])
    q = [min(case["q_max"] if i == 0 or case["q_max"] == 1 else int(r.randint(1, case["q_max"] + 1)), n)
         for i, n in enumerate(lens)]
    if case["op"] == "prefix":
        shared = _groups(case)[1]
        lens = [n + p for n, p in zip(lens, shared)]
    return q, lens


def _groups(case):
    """Where groups of sequences start and end, and the shared keys of each sequence's group: whole pages."""
    b, g = case["batch"], case["groups"]
    cu = [b * i // g for i in range(g + 1)]
    each = [max(1, int(case["prefix"] / (1 + 0.4 * i)) // case["page"]) * case["page"] for i in range(g)]
    return cu, [each[i] for i in range(g) for _ in range(cu[i + 1] - cu[i])], each


def _capacity(case):
    """Rows of a step: what the requests need and a few more, as a program with fixed sizes has."""
    n = sum(_lengths(case)[0])
    return n + 7 - (n + 7) % 8


def _visible(case):
    """Pairs (query, key) that the mask leaves, and the keys that have to be read, over all sequences."""
    pairs = keys = 0
    for q, n in zip(*_lengths(case)):
        p = np.arange(n - q, n, dtype=np.int64)
        first = np.maximum(0, p - case["window"] + 1) if case.get("window") else np.zeros_like(p)
        pairs += int((p - first + 1 + np.minimum(first, case.get("sinks", 0))).sum())
        keys += n - int(first[0]) + min(int(first[0]), case.get("sinks", 0))
    if case["op"] == "prefix":  # a group's shared keys are read once
        cu, shared, each = _groups(case)
        keys += sum(each) - sum(shared)
    return pairs, keys


def _row_bytes(case):
    """Bytes of one token's one head in the cache."""
    b = case["bits"]
    return case["d"] * b / 8 + (case["d"] / 32 if b < 16 else 0)


def work(case):
    if case["op"] == "tables":
        q, kv = _lengths(case)
        p = case["page"]
        new = sum(-(-(a + n) // p) - -(-n // p) for a, n in zip(q, kv))
        # lengths in and out, positions and slots, and the pages' numbers taken and put down
        return {"bytes": 4.0 * (5 * len(q) + 2 * _capacity(case) + 2 * new), "flops": 4.0 * _capacity(case)}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rows":
        t = case["tokens"]
        moved = t * ((hq + hkv) * d * 4 + case["rot"] * 4 + 4 * case["axes"])
        if case["bits"]:  # k is not returned; k and v are written as codes, and read back
            moved += t * hkv * (4 * _row_bytes(case) + 2 * d + 2 * d)
        return {"bytes": moved, "flops": t * (hq + hkv) * (3.0 * case["rot"] + (4.0 * d if case["norm"] else 0))}
    pairs, keys = _visible(case)
    tokens = sum(_lengths(case)[0])
    kv = 2 * d if case["op"] == "prompt" else _row_bytes(case)
    return {"bytes": 2 * keys * hkv * kv + 4 * tokens * hq * d, "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

POSITIONS = 32768


def _axis_of_pair(case):
    """The axis that turns each pair: blocks of pairs, or the axes in turn."""
    half = case["rot"] // 2
    n = case["axes"]
    return [i % n for i in range(half)] if case["cycle"] else [i * n // half for i in range(half)]


def _angles(case):
    """cos and sin [positions, rot/2], float32 from 64-bit angles."""
    half = case["rot"] // 2
    inv = 1e6 ** -(torch.arange(half, dtype=torch.float64, device=DEV) / half)
    a = torch.arange(POSITIONS, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def _quantise(x, dtype, bits):
    """Codes (as the e4m3 or e2m1 values they stand for, and their bytes) and scale bytes of x [..., d]."""
    f = x.float()
    lo, hi = SCALE_RANGE[(dtype, bits)]
    top, fits = (448.0, 448.0) if bits == 8 else (6.0, 7.0)
    blocks = f.reshape(*f.shape[:-1], f.shape[-1] // 32, 32)
    amax = blocks.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax / fits)  # amax / fits = m * 2^e, 0.5 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax == 0, torch.full_like(e, lo), e.clamp(lo, hi))
    y = torch.ldexp(blocks, -e).clamp(-top, top)
    scale = (e + 127).to(torch.uint8).squeeze(-1)
    if bits == 8:
        code = y.to(torch.float8_e4m3fn).reshape(f.shape)
        return code.view(torch.uint8), scale
    grid = torch.tensor(E2M1, device=f.device)
    # the number of midpoints below |y|; a value at a midpoint goes to the even code
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    code += (a > mid[0])
    code += (a >= mid[1])
    code += (a > mid[2])
    code += (a >= mid[3])
    code += (a > mid[4])
    code += (a >= mid[5])
    code += (a > mid[6])
    code = (code | ((y.view(torch.int32) >> 28) & 8).to(torch.uint8)).reshape(f.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(code, scale, bits, wide=torch.float32):
    """The values that codes and scales stand for."""
    if bits == 8:
        v = code.view(torch.float8_e4m3fn).to(wide)
    else:
        grid = torch.tensor(E2M1 + tuple(-g for g in E2M1), dtype=wide, device=code.device)
        v = grid[torch.stack((code & 15, code >> 4), -1).reshape(*code.shape[:-1], 2 * code.shape[-1]).int()]
    return torch.ldexp(v.reshape(*scale.shape, 32), scale[..., None].int() - 127).to(wide).reshape(v.shape)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 23)
    return g


def _keys(shape, g, dtype):
    """Keys as layers give them: some channels of a head far larger than the others."""
    gain = torch.exp2(torch.randn(shape[-2:], generator=g, device=DEV))
    return (torch.randn(shape, generator=g, device=DEV) * gain).to(DTYPES[dtype])


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(DTYPES[dtype])


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "tables":
        _prepare_tables(case, s, g)
    elif case["op"] == "rows":
        _prepare_rows(case, s, g)
    else:
        _prepare_attention(case, s, g)
    if own:  # the handles that a program keeps
        import linear_exl3_input_amd as ex
        if "table" in s:
            s["rope"] = ex.Rope(s["table"], interleaved=case["interleaved"],
                                axes=_axis_of_pair(case) if case["axes"] > 1 else None)
            s["norm"] = ex.HeadNorm(s["wq"], s["wk"], EPS) if case["norm"] else None
        if "ck" in s:
            s["cache"] = ex.KvCache(s["ck"], s["cv"], s["ks"], s["vs"], dtype=DTYPES[case["dtype"]])
        if case["op"] == "tables":
            s["pool"] = ex.KvCache.empty(s["n_pages"], case["page"], 1, 64, 4)
    return s


def _prepare_tables(case, s, g):
    q, kv = _lengths(case)
    page = case["page"]
    have = [-(-n // page) for n in kv]
    more = [-(-(a + n) // page) - h for a, n, h in zip(q, kv, have)]
    s["n_pages"] = sum(have) + sum(more) + 5
    order = torch.randperm(s["n_pages"], generator=g, device=DEV).int()
    width = -(-(case["kv_max"] + case["q_max"]) // page)
    pages = torch.full((len(q), width), -1, dtype=torch.int32, device=DEV)
    pages[torch.arange(width, device=DEV)[None] < _ints(have)[:, None]] = order[:sum(have)]
    # the batch's order is another one for every seed
    at = torch.randperm(len(q), generator=g, device=DEV)
    s["pages"], s["free"] = pages[at].contiguous(), order[sum(have):].contiguous()
    s["q_len"], s["kv_len"] = _ints(q)[at].contiguous(), _ints(kv)[at].contiguous()
    s["rows"] = _capacity(case)


def _prepare_rows(case, s, g):
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], case["dtype"]
    # one projection's output: q, k and v are views of it
    qkv = _normal((t, (hq + 2 * hkv) * d), g, dt)
    s["q"] = qkv[:, :hq * d].view(t, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    s["table"] = _angles(case)
    s["pos"] = torch.randint(0, POSITIONS, (t,), generator=g, device=DEV, dtype=torch.int32)
    if case["axes"] > 1:  # frames of 24 x 40 patches after each other, from a random start
        at = torch.arange(t, device=DEV) + int(torch.randint(0, 960, (1,), generator=g, device=DEV))
        start = int(torch.randint(0, POSITIONS // 2, (1,), generator=g, device=DEV))
        s["pos"] = torch.stack((at // 960, at // 40 % 24, at % 40)[-case["axes"]:]).add(start).int()
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(DTYPES[dt]) for _ in range(2))
    if case["bits"]:
        pages = -(-t // case["page"]) + 3
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=DEV)[:t].int()
        if t > 512:  # tokens of a prompt lie one after another in their pages
            order = torch.randperm(pages, generator=g, device=DEV)
            at = torch.arange(t, device=DEV)
            s["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).int()
        s.update(_cache(case, pages))


def _prepare_attention(case, s, g):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], case["dtype"]
    qs, lens = _lengths(case)
    t = sum(qs)
    s["cu"] = _ints([0] + list(np.cumsum(qs)))
    s["seq"] = torch.repeat_interleave(torch.arange(len(qs), device=DEV), torch.tensor(qs, device=DEV))
    s["q"] = _normal((t, hq, d), g, dt)
    if case["op"] == "prompt":
        s["k"], s["v"] = _normal((t, hkv, d), g, dt), _normal((t, hkv, d), g, dt)
        return
    page = case["page"]
    per = [-(-n // page) for n in lens]
    width = max(per)
    at = torch.arange(width, device=DEV)[None]
    used = at < _ints(per)[:, None]
    if case["op"] == "prefix":
        cu, shared, each = _groups(case)
        of = torch.repeat_interleave(torch.arange(len(each), device=DEV), torch.tensor(np.diff(cu), device=DEV))
        mine = used & (at >= _ints(shared)[:, None] // page)
        n_shared = sum(each) // page
    elif case["freed"]:  # pages that no new token sees are not the sequence's any more
        first = _ints([max(0, n - q - case["window"] + 1) for q, n in zip(qs, lens)])[:, None]
        mine = used & ((at * page < case["sinks"]) | ((at + 1) * page > first))
    else:
        mine = used
    n_mine = int(mine.sum())
    pages = n_mine + (n_shared if case["op"] == "prefix" else 0) + 2
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[mine] = order[:n_mine]
    if case["op"] == "prefix":
        start = torch.tensor(np.cumsum([0] + each[:-1]) // page, device=DEV)[of]
        theirs = at < _ints(shared)[:, None] // page
        table[theirs] = order[n_mine + (start[:, None] + at)[theirs]]
        s["group_cu"], s["prefix_len"] = _ints(cu), _ints(each)
    s["pages"], s["kv_len"] = table, _ints(lens)
    # where each new token stands in a [sequence, new token] array
    s["tok"] = torch.arange(t, device=DEV) - s["cu"][s["seq"]]
    s.update(_cache(case, pages, g))


def _cache(case, pages, g=None):
    """The cache's tensors, empty or holding keys and values."""
    hkv, d, bits, dt, page = case["hkv"], case["d"], case["bits"], case["dtype"], case["page"]
    shape = (pages, hkv, page, d)
    if bits == 16:
        if g is None:
            return dict(ck=torch.zeros(shape, dtype=DTYPES[dt], device=DEV),
                        cv=torch.zeros(shape, dtype=DTYPES[dt], device=DEV), ks=None, vs=None)
        return dict(ck=_keys((pages, page, hkv, d), g, dt).transpose(1, 2).contiguous(), cv=_normal(shape, g, dt),
                    ks=None, vs=None)
    if g is None:
        z = lambda n: torch.zeros((*shape[:-1], n), dtype=torch.uint8, device=DEV)  # noqa: E731
        return dict(ck=z(d * bits // 8), cv=z(d * bits // 8), ks=z(d // 32), vs=z(d // 32))
    ck, ks = _quantise(_keys((pages, page, hkv, d), g, dt).transpose(1, 2).contiguous(), dt, bits)
    cv, vs = _quantise(_normal(shape, g, dt), dt, bits)
    return dict(ck=ck, cv=cv, ks=ks, vs=vs)


# --------------------------------------------------------------- plain form

def _plain_tables(s):
    page, rows, table = s["case"]["page"], s["rows"], s["pages"]
    batch, width = table.shape
    total = s["q_len"].cumsum(0)
    off = (total - s["q_len"]).clamp_max(rows)
    cu = torch.cat((off, total[-1:].clamp_max(rows)))
    kept = cu[1:] - off
    after = s["kv_len"] + kept
    have, need = ((n + page - 1).div(page, rounding_mode="floor").clamp_max(width) for n in (s["kv_len"], after))
    taken = (need - have).cumsum(0)
    at = torch.arange(width, device=DEV)[None]
    index = (taken - (need - have))[:, None] + at - have[:, None]
    fresh = torch.where(index < len(s["free"]), s["free"][index.clamp(0, len(s["free"]) - 1)], -1)
    table = torch.where((at >= have[:, None]) & (at < need[:, None]), fresh, table)
    row = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    used = seq < batch
    seq = seq.clamp_max(batch - 1)
    pos = torch.where(used, s["kv_len"][seq] + row - cu[seq], 0)
    at = pos.div(page, rounding_mode="floor")
    own_page = table[seq, at.clamp_max(width - 1)]
    missing = ~used | (at >= width) | (own_page < 0) | (own_page >= s["n_pages"])
    slots = torch.where(missing, -1, own_page * page + pos % page)
    counts = torch.stack((total[-1], taken[-1]))
    return cu.int(), after.int(), pos.int(), slots.int(), table, counts.int()


def _normed(x, w):
    f = x.float()
    return f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()


def _turn(f, cs, interleaved, dtype):
    """f [t, h, d] in 32 bits with its first 2*cs.shape[1] dims rotated, rounded to the type."""
    rot = 2 * cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if interleaved:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, f[..., rot:]), -1).to(dtype)


def _plain_rows(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["axes"] > 1:
        axis = torch.tensor(_axis_of_pair(c), device=DEV)
        cs = s["table"][s["pos"][axis].T.long(), torch.arange(len(axis), device=DEV)]
    else:
        cs = s["table"][s["pos"].long()]
    q, k = (_normed(s[n], s["w" + n]) if c["norm"] else s[n].float() for n in "qk")
    q, k = (_turn(x, cs, c["interleaved"], dt) for x in (q, k))
    if not c["bits"]:
        return q, k
    out = [q]
    page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    for x, codes, scales in ((k, s["ck"], s["ks"]), (s["v"], s["cv"], s["vs"])):
        if c["bits"] == 16:
            codes[page, :, off] = x
            out.append(codes[page, :, off])
        else:
            codes[page, :, off], scales[page, :, off] = _quantise(x, c["dtype"], c["bits"])
            out.append(_values(codes[page, :, off], scales[page, :, off], c["bits"]).to(dt))
    return out


def _attend(q, k, v, mask, scale):
    """q [..., g, n, d], k and v [..., 1, m, d] in 32 bits, mask [..., 1, n, m]."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale)
    w.masked_fill_(~mask, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_attention(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    g = c["hq"] // c["hkv"]
    scale = c["d"] ** -0.5
    if c["op"] == "prompt":
        at = torch.arange(len(s["seq"]), device=DEV)
        local = at - s["cu"][s["seq"]]
        mask = (s["seq"][:, None] == s["seq"][None]) & (at[:, None] >= at[None])
        mask &= (at[:, None] - at[None] < c["window"]) | (local < c["sinks"])[None]
        q = s["q"].float().view(len(at), c["hkv"], g, c["d"]).permute(1, 2, 0, 3)
        k, v = (s[n].float().permute(1, 0, 2)[:, None] for n in "kv")
        return _attend(q, k, v, mask, scale).permute(2, 0, 1, 3).reshape(s["q"].shape).to(dt)
    b, width = s["pages"].shape
    table = s["pages"].clamp_min(0).long()
    kv = []
    for codes, scales in ((s["ck"], s["ks"]), (s["cv"], s["vs"])):
        x = codes[table].float() if c["bits"] == 16 else _values(codes[table], scales[table], c["bits"])
        kv.append(x.transpose(1, 2).reshape(b, c["hkv"], 1, width * c["page"], c["d"]))
    n = c["q_max"]
    q = torch.zeros((b, n, c["hq"], c["d"]), device=DEV)
    q[s["seq"], s["tok"]] = s["q"].float()
    q = q.view(b, n, c["hkv"], g, c["d"]).permute(0, 2, 3, 1, 4)
    count = s["cu"][1:] - s["cu"][:-1]
    pos = ((s["kv_len"] - count)[:, None] + torch.arange(n, device=DEV)[None])[..., None]
    at = torch.arange(width * c["page"], device=DEV)
    mask = (at <= pos) & (s["pages"] >= 0).repeat_interleave(c["page"], 1)[:, None]
    if c["op"] == "paged":
        mask &= (at > pos - c["window"]) | (at < c["sinks"])
    o = _attend(q, kv[0], kv[1], mask[:, None, None], scale)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], c["d"])[s["seq"], s["tok"]].to(dt)


def _own(s):
    import linear_exl3_input_amd as ex
    c = s["case"]
    if c["op"] == "tables":
        step = ex.cache_extend(s["pool"], s["q_len"], s["kv_len"], s["pages"], s["free"], s["rows"])
        return step.cu_q, step.kv_len, step.positions, step.slots, s["pages"], step.counts
    if c["op"] == "rows":
        if not c["bits"]:
            return ex.rope(s["rope"], s["pos"], s["q"], s["k"], norm=s["norm"])
        q = ex.rope_cache_write(s["cache"], s["rope"], s["pos"], s["slots"], s["q"], s["k"], s["v"], norm=s["norm"])
        return [q, *ex.cache_read(s["cache"], s["slots"])]
    if c["op"] == "prompt":
        return ex.prompt_attention(s["q"], s["k"], s["v"], s["cu"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "paged":
        return ex.paged_attention(s["cache"], s["q"], s["cu"], s["kv_len"], s["pages"], window=c["window"],
                                  sinks=c["sinks"])
    return ex.prefix_attention(s["cache"], s["q"], s["cu"], s["kv_len"], s["pages"], s["group_cu"], s["prefix_len"])


def run(state):
    if own:
        return _own(state)
    plain = {"tables": _plain_tables, "rows": _plain_rows}
    return plain.get(state["case"]["op"], _plain_attention)(state)


# ------------------------------------------------------------------ 64 bits

def _round16(x, dtype):
    """float64 rounded once to the type (through float32 it could round twice)."""
    bits = 7 if dtype == BF16 else 10
    least = -126 if dtype == BF16 else -14
    _, e = torch.frexp(x)
    e = (e - 1).clamp_min(least) - bits
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


def _exact_turned(x, w, case, table, pos):
    x = x.double().cpu()
    if case["norm"]:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double().cpu()
    pos = pos.cpu().long().reshape(-1, x.shape[0])
    table = table.double().cpu()
    y = x.clone()
    for i, axis in enumerate(_axis_of_pair(case)):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
        c, s = table[pos[axis], i].T[..., None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _exact_quantised(x, dtype, bits):
    """What is read back of x [t, h, d] in 64 bits: each block's values to the nearest of the format's."""
    if bits == 16:
        return x
    lo, hi = SCALE_RANGE[(dtype, bits)]
    t = x.reshape(*x.shape[:-1], -1, 32)
    amax = t.abs().amax(-1, keepdim=True)
    e = torch.full_like(amax, lo)
    for n in range(lo, hi):  # one more for each power of two that does not hold the largest value
        e += (amax > math.ldexp(448.0 if bits == 8 else 7.0, n)).double()
    y = t * torch.exp2(-e)
    top, mantissa, least = (448.0, 3, -6) if bits == 8 else (6.0, 1, 0)
    y = y.clamp(-top, top)
    _, p = torch.frexp(y)
    step = torch.exp2(((p - 1).clamp_min(least) - mantissa).double())
    return (torch.round(y / step) * step * torch.exp2(e)).reshape(x.shape)


def _exact_tables(s):
    page, rows, n_pages = s["case"]["page"], s["rows"], s["n_pages"]
    table, free = s["pages"].tolist(), s["free"].tolist()
    cu, after, pos, slots, taken = [0], [], [], [], 0
    for row, q, kv in zip(table, s["q_len"].tolist(), s["kv_len"].tolist()):
        have = math.ceil(kv / page)
        kept = min(q, rows - cu[-1])
        for i in range(have, min(len(row), math.ceil((kv + kept) / page))):
            row[i] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(kv, kv + kept):
            i = row[p // page] if p // page < len(row) else -1
            pos.append(p)
            slots.append(i * page + p % page if 0 <= i < n_pages else -1)
        cu.append(cu[-1] + kept)
        after.append(kv + kept)
    pad = rows - len(pos)
    counts = [int(s["q_len"].sum()), taken]
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return ints(cu), ints(after), ints(pos + [0] * pad), ints(slots + [-1] * pad), ints(table), ints(counts)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "rows":
        q, k = (_exact_turned(s[n], s["w" + n], case, s["table"], s["pos"]) for n in "qk")
        if not case["bits"]:
            return q, k
        # the cache quantises the rotated keys in their own type
        k = _round16(k, case["dtype"])
        return [q] + [_exact_quantised(x, case["dtype"], case["bits"]) for x in (k, s["v"].double().cpu())]
    qs, lens = _lengths(case)
    g, out, done = case["hq"] // case["hkv"], torch.empty(s["q"].shape, dtype=torch.float64, device=DEV), 0
    for i, (n, m) in enumerate(zip(qs, lens)):
        if case["op"] == "prompt":
            kv = [s[name][done:done + n].double() for name in "kv"]
            held = torch.ones(m, dtype=torch.bool, device=DEV)
        else:
            ids = s["pages"][i][:-(-m // case["page"])].long()
            held = (ids >= 0).repeat_interleave(case["page"])[:m]
            ids = ids.clamp_min(0)
            kv = [(codes[ids].double() if case["bits"] == 16 else
                   _values(codes[ids], scales[ids], case["bits"], torch.float64)).transpose(1, 2).flatten(0, 1)[:m]
                  for codes, scales in ((s["ck"], s["ks"]), (s["cv"], s["vs"]))]
        for h in range(case["hq"]):
            k, v = (x[:, h // g] for x in kv)
            for at in range(0, n, 2048):  # rows
                rows = min(2048, n - at)
                w = s["q"][done + at:done + at + rows, h].double() @ k.T / math.sqrt(case["d"])
                key = torch.arange(m, device=DEV)
                gap = torch.arange(m - n + at, m - n + at + rows, device=DEV)[:, None] - key
                seen = (gap >= 0) & held
                if "window" in case:
                    seen &= (gap < case["window"]) | (key < case["sinks"])
                out[done + at:done + at + rows, h] = torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ v
        done += n
    return out
