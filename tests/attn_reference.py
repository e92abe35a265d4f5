"""The attention operators' definitions in 64 bits, on the CPU, and the bounds
that a 16-bit result with fp32 sums keeps to.  Shares no code with the
package.  Not collected by pytest."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# exponents of a block's scale: (least, greatest), see include/exl3_attn.h
RANGE = {(torch.bfloat16, 8): (-117, 119), (torch.bfloat16, 4): (-125, 125),
         (torch.float16, 8): (-15, 7), (torch.float16, 4): (-23, 13)}


def unit(dtype):
    """Largest relative error of one rounding to nearest."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11


def smallest(dtype):
    """Half the spacing of the type's subnormals (bf16's are below anything here)."""
    return 0.0 if dtype == torch.bfloat16 else 2.0 ** -25


# ------------------------------------------------------------------- rotary

def rotate(x, table, pos, interleaved):
    """(value, bound of an fp32 evaluation rounded once) of x [t, h, d]."""
    x64, cs = x.double(), table.double()[pos.long()][:, None]
    half = table.shape[1]
    a = x64[..., 0:2 * half:2] if interleaved else x64[..., :half]
    b = x64[..., 1:2 * half:2] if interleaved else x64[..., half:2 * half]
    c, s = cs[..., 0], cs[..., 1]
    ra, rb = a * c - b * s, b * c + a * s
    ma, mb = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    y, mag = x64.clone(), torch.zeros_like(x64)
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
        mag[..., 0:2 * half:2], mag[..., 1:2 * half:2] = ma, mb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
        mag[..., :half], mag[..., half:2 * half] = ma, mb
    # two products and a sum in fp32: 2 roundings of 2^-24 on each term
    f32 = 2.01 * 2.0 ** -24 * mag
    bound = torch.where(mag > 0, unit(x.dtype) * (y.abs() + f32) + f32 + smallest(x.dtype), torch.zeros_like(mag))
    return y, bound


# -------------------------------------------------------------------- cache

def quantise(x, bits):
    """What a cache of `bits` reads back of x [..., d] (16-bit type), in float64: exact, since
    scaling by powers of two and rounding to a grid are."""
    if bits == 16:
        return x.double()
    lo, hi = RANGE[(x.dtype, bits)]
    top, fits = (448.0, 448.0) if bits == 8 else (6.0, 7.0)
    v = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(v).all(-1, keepdim=True)
    safe = torch.where(bad, torch.ones_like(amax), amax)
    e = torch.full_like(safe, lo)
    for n in range(lo, hi):
        e += (safe > fits * 2.0 ** n).double()
    y = (v * torch.exp2(-e)).clamp(-top, top)
    if bits == 4:
        grid = torch.tensor(E2M1, dtype=torch.float64)
        gap = (y.abs()[..., None] - grid).abs()
        near = gap.amin(-1, keepdim=True)
        # of two equally near, the even code (an even place in the grid)
        order = gap + torch.arange(8) % 2 * 1e-9
        order = torch.where(gap == near, order, torch.full_like(order, 9.0))
        q = grid[order.argmin(-1)] * torch.where(y < 0, -1.0, 1.0)
    else:
        _, p = torch.frexp(y)
        step = torch.exp2(((p - 1).clamp_min(-6) - 3).double())
        q = torch.round(y / step) * step
    out = torch.where(bad, torch.full_like(q, math.nan), q * torch.exp2(e))
    return out.reshape(x.shape)


# ---------------------------------------------------------------- attention

def attend(q, k, v, seen, scale, dtype):
    """(value, bound) of one sequence: q [n, hq, d], k and v [m, hkv, d] in float64, seen [n, m] bool.  Each row is
    computed over the keys it sees alone, so nothing that it does not see can reach it."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.zeros(n, hq, v.shape[-1], dtype=torch.float64)
    bound = torch.zeros_like(out)
    u = unit(dtype)
    for i in range(n):
        idx = seen[i].nonzero()[:, 0]
        if len(idx) == 0:
            continue
        ki = k[idx].repeat_interleave(g, 1)  # [m', hq, d]
        vi = v[idx].repeat_interleave(g, 1)
        s = torch.einsum("hd,mhd->hm", q[i], ki) * scale
        mag = torch.einsum("hd,mhd->hm", q[i].abs(), ki.abs()) * scale
        p = torch.softmax(s, -1)
        out[i] = torch.einsum("hm,mhd->hd", p, vi)
        a = torch.einsum("hm,mhd->hd", p, vi.abs())
        # a score's error: d products and sums in fp32 and three more roundings; a probability's: that twice (its own
        # and the maximum's or the sum's), a few roundings of exp2, products and sums, and its own to the type
        delta = 2 * (d + 4) * 2.0 ** -23 * mag.amax(-1, keepdim=True) + (len(idx) + 64) * 2.0 ** -23
        err = (u + delta) * 1.01 * a + smallest(dtype) * vi.abs().sum(0)
        bound[i] = u * (out[i].abs() + err) + err + smallest(dtype)
    return out, bound


def mask(q_len, kv_len, causal=True, window=0, page_table=None, page_size=0, pages=0):
    """seen [q_len, kv_len] of one sequence."""
    if q_len == 0 or kv_len == 0:
        return torch.zeros(q_len, kv_len, dtype=torch.bool)
    gap = torch.arange(kv_len - q_len, kv_len)[:, None] - torch.arange(kv_len)
    seen = torch.ones(q_len, kv_len, dtype=torch.bool) if not causal else gap >= 0
    if window:
        seen = seen & (gap < window)
    if page_table is not None:
        at = torch.arange(kv_len) // page_size
        have = at < len(page_table)
        pg = torch.where(have, page_table[at.clamp_max(max(0, len(page_table) - 1))].long(), -1) if len(page_table) else \
            torch.full((kv_len,), -1)
        seen = seen & ((pg >= 0) & (pg < pages))
    return seen


def check(got, want, bound, what):
    """Every element within its bound; a value that is not finite must be the same kind of value."""
    got = got.double().cpu()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: {int((torch.isfinite(got) != fin).sum())} values differ in being finite"
    # infinities and NaN: a NaN where the definition has one or the sum of opposite infinities, else the same infinity
    assert torch.equal(torch.isnan(got[~fin]), torch.isnan(want[~fin])), f"{what}: NaN against infinity"
    both = ~fin & ~torch.isnan(want)
    assert torch.equal(got[both], want[both]), f"{what}: infinities of other signs"
    over = ((got - want).abs() - bound)[fin]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} values outside the bound, worst by {worst:.3e}"
