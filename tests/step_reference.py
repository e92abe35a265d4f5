"""The definitions of the step's operators (include/exl3_step.h) in 64 bits and
whole numbers, on the CPU, and the bounds that fp32 evaluations rounded once
keep to.  Shares no code with the package.  Not collected by pytest."""
import torch

import attn_reference as ref


def normed(x, weight, eps):
    """(value, bound of the fp32 evaluation) of x [t, h, d] normed per head; weight [d] or [h, d]."""
    x64 = x.double()
    y = x64 / torch.sqrt(x64.square().mean(-1, keepdim=True) + eps) * weight.double()
    # the sum of squares: a rounding for each square and at most 14 sums after each other (8 values a lane, then lanes
    # in pairs), the sum with eps: 16 of 2^-24, of which the root takes half; the root itself 2^-23; two products
    return y, (8 + 2 + 2) * 1.01 * 2.0 ** -24 * y.abs()


def turned(x, err, table, positions, axes, interleaved, dtype):
    """(value, bound) of x [t, h, d] in 64 bits, known to err, with pair i turned by positions[axes[i]] and rounded."""
    half = table.shape[1]
    pos = positions.reshape(-1, x.shape[0]).long()
    cs = torch.stack([table.double()[pos[a], i] for i, a in enumerate(axes)], 1)[:, None]  # [t, 1, half, 2]
    c, s = cs[..., 0], cs[..., 1]

    def split(v):
        return (v[..., 0:2 * half:2], v[..., 1:2 * half:2]) if interleaved else (v[..., :half], v[..., half:2 * half])

    def join(whole, a, b):
        whole = whole.clone()
        if interleaved:
            whole[..., 0:2 * half:2], whole[..., 1:2 * half:2] = a, b
        else:
            whole[..., :half], whole[..., half:2 * half] = a, b
        return whole

    (a, b), (ea, eb) = split(x), split(err)
    y = join(x, a * c - b * s, b * c + a * s)
    mag = join(torch.zeros_like(x), (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())
    off = join(err, ea * c.abs() + eb * s.abs(), eb * c.abs() + ea * s.abs())
    # two products and a sum in fp32: 2 roundings on each term
    f32 = (2.01 * 2.0 ** -24 * mag + off) * 1.01
    changed = (mag > 0) | (err > 0)
    bound = ref.unit(dtype) * (y.abs() + f32) + f32 + ref.smallest(dtype)
    return y, torch.where(changed, bound, torch.zeros_like(bound))


def extended(pages, page_size, q_len, kv_len, table, free, tokens, taken=0):
    """(cu_q, kv_out, positions, slots, counts, table) as lists, one row after another."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    cu, out, pos, slots, need = [0], [], [], [], 0
    taken = min(max(taken, 0), len(free))
    wanted = 0
    for row, q, kv in zip(table, q_len, kv_len):
        q, kv = min(max(q, 0), 1 << 20), min(max(kv, 0), 1 << 30)
        wanted += q
        kept = min(q, tokens - cu[-1])
        for i in range(min(width, -(-kv // page_size)), min(width, -(-(kv + kept) // page_size))):
            row[i] = free[taken + need] if taken + need < len(free) else -1
            need += 1
        for p in range(kv, kv + kept):
            page = row[p // page_size] if p // page_size < width else -1
            pos.append(p)
            slots.append(page * page_size + p % page_size if 0 <= page < pages else -1)
        cu.append(cu[-1] + kept)
        out.append(kv + kept)
    pad = tokens - len(pos)
    return cu, out, pos + [0] * pad, slots + [-1] * pad, [min(wanted, 2 ** 31 - 1), need], table
