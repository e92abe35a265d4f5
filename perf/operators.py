"""The work of the attention operators: rotary positions, the quantised paged
cache, attention over that cache and attention over packed prompts.

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

# The least and greatest exponent of a block's scale: every stored value is
# then exact in the cache's 16-bit type.
SCALE_RANGE = {(BF16, 8): (-117, 119), (BF16, 4): (-125, 125), (F16, 8): (-15, 7), (F16, 4): (-23, 13)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One step of 16 sequences: q and k of a layer with 256-wide heads of which a quarter turns.
        dict(name="rope_step", op="rope", tokens=16, hq=24, hkv=4, d=256, rot=64, interleaved=False, dtype=BF16,
             positions=32768, factor=1.0),
        # A prompt of odd length, interleaved pairs over the whole head, positions scaled for a long context.
        dict(name="rope_prompt", op="rope", tokens=4099, hq=32, hkv=8, d=128, rot=128, interleaved=True, dtype=F16,
             positions=131072, factor=4.0),
        # One step of 48 sequences, rotated and written to a 4-bit cache in one call, and read back.
        dict(name="write_step_4bit", op="store", tokens=48, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype=BF16, bits=4, page=64, fused=True, positions=32768),
        # A long prompt's keys and values written to an 8-bit cache and read back.
        dict(name="write_prompt_8bit", op="store", tokens=16300, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype=BF16, bits=8, page=32, fused=False, positions=32768),
        # One sequence, one new token, a short context: the latency of a chat's step.
        dict(name="paged_single", op="paged", batch=1, q_max=1, kv_max=1100, hq=32, hkv=8, d=128, dtype=BF16, bits=16,
             page=64, window=0),
        # A busy server's step: 64 sequences of very different lengths, 8-bit cache.
        dict(name="paged_batch_8bit", op="paged", batch=64, q_max=1, kv_max=16000, hq=32, hkv=8, d=128, dtype=BF16,
             bits=8, page=64, window=0),
        # A few very long contexts in a 4-bit cache, wide heads.
        dict(name="paged_long_4bit", op="paged", batch=3, q_max=1, kv_max=120000, hq=24, hkv=4, d=256, dtype=BF16,
             bits=4, page=128, window=0),
        # Checking drafted tokens: a few new tokens of each sequence, a window, narrow heads.
        dict(name="paged_draft", op="paged", batch=24, q_max=7, kv_max=9000, hq=64, hkv=8, d=64, dtype=F16, bits=16,
             page=16, window=4096),
        # Chunks of prompts continued over what is cached.
        dict(name="paged_chunk_8bit", op="paged", batch=3, q_max=1000, kv_max=20000, hq=32, hkv=8, d=128, dtype=BF16,
             bits=8, page=64, window=0),
        # Many short prompts packed together, narrow heads.
        dict(name="prompt_short", op="prompt", batch=20, len_max=300, hq=16, hkv=4, d=64, dtype=F16, window=0),
        # Prompts of different lengths packed together, the longest 8000 tokens.
        dict(name="prompt_long", op="prompt", batch=3, len_max=8000, hq=32, hkv=8, d=128, dtype=BF16, window=0),
        # Wide heads, a sliding window.
        dict(name="prompt_wide", op="prompt", batch=2, len_max=5000, hq=24, hkv=4, d=256, dtype=BF16, window=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "store", "paged", "paged", "prompt"))
    d = rng.choice((64, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 6, 8))
    case = dict(op=op, hq=hq, hkv=hkv, d=d, dtype=rng.choice((BF16, F16)))
    if op in ("rope", "store"):
        case.update(rot=rng.choice((d // 4, d // 2, d)), interleaved=rng.random() < 0.5, tokens=_log(rng, 1, 8000),
                    positions=rng.choice((32768, 131072)))
    if op == "rope":
        case.update(factor=rng.choice((1.0, 4.0, 8.0)))
    if op == "store":
        case.update(bits=rng.choice((16, 8, 4)), page=rng.choice((16, 32, 64, 128, 256)), fused=rng.random() < 0.5)
    if op == "paged":
        q = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 700)))
        batch = _log(rng, 1, 64 if q <= 16 else 4)
        case.update(bits=rng.choice((16, 8, 4)), page=rng.choice((16, 32, 64, 128, 256)), batch=batch, q_max=q,
                    kv_max=max(q, _log(rng, 16, 60000 if batch <= 8 and q <= 16 else 12000)),
                    window=rng.choice((0, 0, _log(rng, 100, 4096))))
    if op == "prompt":
        batch = _log(rng, 1, 24)
        case.update(batch=batch, len_max=_log(rng, 2, 6000 // max(1, batch // 2)),
                    window=rng.choice((0, 0, _log(rng, 100, 4096))))
    return case


def _lengths(case):
    """The lengths of a case's sequences: the first as long as stated, the
    others spread from very short to that, the same for every seed."""
    r = np.random.RandomState(1234 + case["batch"])
    top = case["kv_max"] if case["op"] == "paged" else case["len_max"]
    lens = [top] + [max(1, int(top * r.uniform(0.02, 1.0) ** 1.5)) for _ in range(case["batch"] - 1)]
    if case["op"] == "prompt":
        return lens, lens
    q = [min(case["q_max"] if i == 0 or case["q_max"] == 1 else int(r.randint(1, case["q_max"] + 1)), n)
         for i, n in enumerate(lens)]
    return q, lens


def _visible(case):
    """Pairs (query, key) that the mask leaves, and the keys that some query sees, over all sequences."""
    pairs = keys = 0
    for q, n in zip(*_lengths(case)):
        p = np.arange(n - q, n, dtype=np.int64)
        first = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        pairs += int((p - first + 1).sum())
        keys += n - int(first[0])
    return pairs, keys


def _row_bytes(case):
    """Bytes of one token's one head in the cache."""
    b = case["bits"]
    return case["d"] * b / 8 + (case["d"] / 32 if b < 16 else 0)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": t * ((hq + hkv) * d * 4 + case["rot"] * 4 + 4), "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    if case["op"] == "store":
        t = case["tokens"]
        kv = 2 * t * hkv * (2 * d + _row_bytes(case))  # written: values read, codes written
        back = 2 * t * hkv * (2 * d + _row_bytes(case))  # read back: the reverse
        q = t * (hq * d * 4 + case["rot"] * 4) if case["fused"] else 0
        return {"bytes": kv + back + q, "flops": 6.0 * t * hkv * d + (3.0 * t * hq * case["rot"] if case["fused"] else 0)}
    pairs, keys = _visible(case)
    tokens = sum(_lengths(case)[0])
    kv = _row_bytes(case) if case["op"] == "paged" else 2 * d
    return {"bytes": 2 * keys * hkv * kv + 4 * tokens * hq * d, "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _angles(case):
    """cos and sin [positions, rot/2], with the frequencies of a context that
    was stretched by `factor`: slow pairs divided by it, fast ones kept, a
    ramp between; float32 from 64-bit angles."""
    half = case["rot"] // 2
    inv = 1e6 ** -(torch.arange(half, dtype=torch.float64, device=DEV) / half)
    turns = case["positions"] / case.get("factor", 1.0) * inv / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    inv = inv * (keep + (1 - keep) / case.get("factor", 1.0))
    a = torch.arange(case["positions"], dtype=torch.float64, device=DEV)[:, None] * inv
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
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _keys(shape, g, dtype):
    """Keys as layers give them: some channels of a head far larger than the others."""
    gain = torch.exp2(torch.randn(shape[-2:], generator=g, device=DEV))
    return (torch.randn(shape, generator=g, device=DEV) * gain).to(DTYPES[dtype])


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(DTYPES[dtype])


def prepare(case, seed):
    g = _gen(seed)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], case["dtype"]
    s = {"case": case}
    if case["op"] in ("rope", "store"):
        t = case["tokens"]
        # one projection's output: q, k and v are views of it
        qkv = _normal((t, (hq + 2 * hkv) * d), g, dt)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["table"] = _angles(case)
        s["pos"] = torch.randint(0, case["positions"], (t,), generator=g, device=DEV, dtype=torch.int32)
    if case["op"] == "store":
        pages = -(-t // case["page"]) + 3
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=DEV)[:t].int()
        if t > 1:  # tokens of a prompt lie one after another in their pages
            order = torch.randperm(pages, generator=g, device=DEV)
            at = torch.arange(t, device=DEV)
            s["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).int()
        s.update(_cache(case, pages))
    if case["op"] == "prompt":
        lens = _lengths(case)[1]
        t = sum(lens)
        s["q"], s["k"], s["v"] = _normal((t, hq, d), g, dt), _normal((t, hkv, d), g, dt), _normal((t, hkv, d), g, dt)
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        s["seq"] = torch.repeat_interleave(torch.arange(len(lens), device=DEV), torch.tensor(lens, device=DEV))
    if case["op"] == "paged":
        qs, lens = _lengths(case)
        per = [-(-n // case["page"]) for n in lens]
        pages = sum(per) + 2
        order = torch.randperm(pages, generator=g, device=DEV).int()
        table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device=DEV)
        used = torch.arange(max(per), device=DEV)[None] < torch.tensor(per, device=DEV)[:, None]
        table[used] = order[:sum(per)]
        s["pages"], s["kv_len"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu"] = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=DEV)
        s["q"] = _normal((sum(qs), hq, d), g, dt)
        # where each new token stands in a [sequence, new token] array
        s["seq"] = torch.repeat_interleave(torch.arange(len(qs), device=DEV), torch.tensor(qs, device=DEV))
        s["tok"] = torch.arange(sum(qs), device=DEV) - s["cu"][s["seq"]]
        s.update(_cache(case, pages, g))
    if own:  # the handles that a program keeps
        import linear_exl3_input_amd as ex
        if "table" in s:
            s["rope"] = ex.Rope(s["table"], interleaved=case["interleaved"])
        if "ck" in s:
            s["cache"] = ex.KvCache(s["ck"], s["cv"], s["ks"], s["vs"], dtype=DTYPES[dt])
    return s


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

def _turn(x, cs, interleaved):
    """x [t, h, d] with its first 2*cs.shape[1] dims rotated, in x's type."""
    f = x.float()
    rot = 2 * cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if interleaved:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, f[..., rot:]), -1).to(x.dtype)


def _attend(q, k, v, mask, scale):
    """q [..., g, n, d], k and v [..., 1, m, d] in 32 bits, mask [..., 1, n, m]."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale)
    w.masked_fill_(~mask, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    g = c["hq"] // c["hkv"]
    if c["op"] == "rope":
        cs = s["table"][s["pos"].long()]
        return _turn(s["q"], cs, c["interleaved"]), _turn(s["k"], cs, c["interleaved"])
    if c["op"] == "store":
        out, k = [], s["k"]
        if c["fused"]:
            cs = s["table"][s["pos"].long()]
            out, k = [_turn(s["q"], cs, c["interleaved"])], _turn(k, cs, c["interleaved"])
        page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
        for x, codes, scales in ((k, s["ck"], s["ks"]), (s["v"], s["cv"], s["vs"])):
            if c["bits"] == 16:
                codes[page, :, off] = x
                out.append(codes[page, :, off])
            else:
                codes[page, :, off], scales[page, :, off] = _quantise(x, c["dtype"], c["bits"])
                out.append(_values(codes[page, :, off], scales[page, :, off], c["bits"]).to(dt))
        return out
    scale = c["d"] ** -0.5
    if c["op"] == "prompt":
        at = torch.arange(len(s["seq"]), device=DEV)
        mask = (s["seq"][:, None] == s["seq"][None]) & (at[:, None] >= at[None])
        if c["window"]:
            mask &= at[:, None] - at[None] < c["window"]
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
    pos = (s["kv_len"] - count)[:, None] + torch.arange(n, device=DEV)[None]
    at = torch.arange(width * c["page"], device=DEV)
    mask = at <= pos[..., None]
    if c["window"]:
        mask &= at > pos[..., None] - c["window"]
    o = _attend(q, kv[0], kv[1], mask[:, None, None], scale)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], c["d"])[s["seq"], s["tok"]].to(dt)


def _own(s):
    import linear_exl3_input_amd as ex
    c = s["case"]
    if c["op"] == "rope":
        return ex.rope(s["rope"], s["pos"], s["q"], s["k"])
    if c["op"] == "store":
        out = []
        if c["fused"]:
            out.append(ex.rope_cache_write(s["cache"], s["rope"], s["pos"], s["slots"], s["q"], s["k"], s["v"]))
        else:
            ex.cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return out + list(ex.cache_read(s["cache"], s["slots"]))
    if c["op"] == "prompt":
        return ex.prompt_attention(s["q"], s["k"], s["v"], s["cu"], window=c["window"])
    return ex.paged_attention(s["cache"], s["q"], s["cu"], s["kv_len"], s["pages"], window=c["window"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _round16(x, dtype):
    """float64 rounded once to the type (through float32 it could round twice)."""
    bits = 7 if dtype == BF16 else 10
    least = -126 if dtype == BF16 else -14
    _, e = torch.frexp(x)
    e = (e - 1).clamp_min(least) - bits
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


def _exact_turn(x, case, table, pos):
    x = x.double().cpu()
    cs = table.double().cpu()[pos.long().cpu()]
    y = x.clone()
    for i in range(case["rot"] // 2):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
        c, s = cs[:, i, 0, None], cs[:, i, 1, None]
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["q"], case, s["table"], s["pos"]), _exact_turn(s["k"], case, s["table"], s["pos"])
    if case["op"] == "store":
        out, k = [], s["k"].double().cpu()
        if case["fused"]:
            out = [_exact_turn(s["q"], case, s["table"], s["pos"])]
            # the cache quantises the rotated keys in their own type
            k = _round16(_exact_turn(s["k"], case, s["table"], s["pos"]), case["dtype"])
        return out + [_exact_quantised(x, case["dtype"], case["bits"]) for x in (k, s["v"].double().cpu())]
    qs, lens = _lengths(case)
    g, out, done = case["hq"] // case["hkv"], torch.empty(s["q"].shape, dtype=torch.float64, device=DEV), 0
    for i, (n, m) in enumerate(zip(qs, lens)):
        if case["op"] == "paged":
            ids = s["pages"][i][:-(-m // case["page"])].long()
            kv = [(codes[ids].double() if case["bits"] == 16 else
                   _values(codes[ids], scales[ids], case["bits"], torch.float64)).transpose(1, 2).flatten(0, 1)[:m]
                  for codes, scales in ((s["ck"], s["ks"]), (s["cv"], s["vs"]))]
        else:
            kv = [s[name][done:done + n].double() for name in "kv"]
        for h in range(case["hq"]):
            k, v = (x[:, h // g] for x in kv)
            for at in range(0, n, 2048):  # rows
                rows = min(2048, n - at)
                w = s["q"][done + at:done + at + rows, h].double() @ k.T / math.sqrt(case["d"])
                gap = torch.arange(m - n + at, m - n + at + rows, device=DEV)[:, None] - torch.arange(m, device=DEV)
                seen = (gap >= 0) & (gap < (case["window"] or m + 1))
                out[done + at:done + at + rows, h] = torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ v
        done += n
    return out
