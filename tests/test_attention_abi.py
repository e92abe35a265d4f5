"""The attention C ABI and its binding on the CPU: exports, sizes, and every
refusal.  No call here reaches a kernel launch (there is no GPU)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
from linear_exl3_input_amd import attention as at

pytestmark = pytest.mark.skipif(not os.path.exists(ex.lib_path()), reason="libexl3.so not built")

FAKE = 0x100000  # a 16-byte aligned address that is never dereferenced
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rows(heads=4, token=None, head=128, data=FAKE):
    return at._Rows(data, heads * 128 if token is None else token, head, heads)


def cache(bits=8, pages=10, page=16, heads=4, d=128, dtype=1, **kw):
    size = heads * page * d * bits // 8
    c = at._Cache(FAKE, FAKE, FAKE if bits < 16 else None, FAKE if bits < 16 else None, size, size,
                  heads * page * d // 32 if bits < 16 else 0, heads * page * d // 32 if bits < 16 else 0, pages, page,
                  heads, d, dtype, bits)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rotary(**kw):
    r = at._Rotary(FAKE, 100, 64, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def last():
    return ex.load().exl3_last_error().decode()


def L():
    return at._lib()


B = ctypes.byref


def test_exports_every_header_symbol():
    names = at.attn_header_symbols()
    assert len(names) == 7
    for name in names:
        assert hasattr(ex.load(), name), name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "a.c"
    src.write_text('#include "exl3_attn.h"\nint main(void) { return sizeof(exl3_kv_cache) == 88 && sizeof(exl3_rows) == 32 '
                   '&& sizeof(exl3_rotary) == 24 ? 0 : 1; }\n')
    exe = str(tmp_path / "a")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0
    assert (ctypes.sizeof(at._Cache), ctypes.sizeof(at._Rows), ctypes.sizeof(at._Rotary)) == (88, 32, 24)


def rope(r=None, tokens=4, d=128, dtype=1, q=None, qo=None, k=None, ko=None, pos=FAKE):
    return L().exl3_rope(B(r or rotary()), pos, tokens, d, dtype, B(q or rows()), B(qo or rows(data=FAKE + 4096 * 64)),
                         B(k) if k else None, B(ko) if ko else None, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(tokens=-1), 1, "tokens=-1 is negative"),
    (dict(tokens=(1 << 20) + 1), 2, "exceeds the supported"),
    (dict(d=96), 2, "head_dim=96"),
    (dict(dtype=2), 1, "dtype=2"),
    (dict(r=rotary(rot=24)), 1, "rot=24"),
    (dict(r=rotary(rot=0)), 1, "rot=0"),
    (dict(r=rotary(rot=144)), 1, "rot=144"),
    (dict(r=rotary(positions=0)), 1, "0 positions"),
    (dict(r=rotary(interleaved=2)), 1, "interleaved=2"),
    (dict(r=rotary(table=None)), 1, "rotary table is NULL"),
    (dict(pos=None), 1, "positions is NULL"),
    (dict(pos=FAKE + 2), 1, "not 4-byte aligned"),
    (dict(q=rows(data=FAKE + 8)), 1, "not 16-byte aligned"),
    (dict(q=rows(token=516)), 1, "multiples of 8"),
    (dict(q=rows(token=-512)), 1, "non-negative"),
    (dict(q=rows(heads=0)), 1, "q has 0 heads"),
    (dict(qo=rows(token=504)), 1, "overlap"),
    (dict(qo=rows(head=64)), 1, "overlap"),
    (dict(qo=rows(token=0)), 1, "overlap"),
    (dict(qo=rows(heads=5)), 1, "q_out has 5 heads, its input 4"),
    (dict(qo=rows(token=1024)), 1, "starts at its input with other strides"),
    (dict(k=rows()), 1, "k and k_out must be given together"),
    (dict(tokens=1 << 20, q=rows(heads=1024, token=1 << 17), qo=rows(heads=1024, token=1 << 17),
          k=rows(heads=1024, token=1 << 17), ko=rows(heads=1024, token=1 << 17)), 2, "exceed 2^31 rows"),
])
def test_rope_refusals(kw, status, msg):
    assert rope(**kw) == status
    assert msg in last()


def test_rope_without_tokens_needs_no_pointers():
    r = at._Rows(None, 0, 0, 4)
    assert rope(tokens=0, q=r, qo=r, pos=None) == 0


@pytest.mark.parametrize("kw,msg", [
    (dict(bits=5), "bits=5"), (dict(page=24), "page_size=24"), (dict(page=8), "page_size=8"),
    (dict(page=2048), "page_size=2048"), (dict(pages=0), "0 pages"), (dict(pages=1 << 28), "must be 1..2^31-1 tokens"),
    (dict(heads=0), "0 heads"), (dict(dtype=7), "dtype=7"), (dict(d=80), "head_dim=80"), (dict(k=None), "cache k is NULL"),
    (dict(v=FAKE + 8), "cache v"), (dict(k_page_bytes=8192 - 16), "k_page_bytes=8176"),
    (dict(v_page_bytes=8200), "v_page_bytes=8200"), (dict(k_scale=None), "cache k_scale is NULL"),
    (dict(v_scale_page_bytes=128), "v_scale_page_bytes=128"), (dict(bits=16, k_scale=FAKE), "no scales"),
])
def test_cache_refusals(kw, msg):
    assert L().exl3_cache_write(B(cache(**kw)), B(rows()), B(rows()), FAKE, 3, None) in (1, 2)
    assert msg in last()
    assert L().exl3_cache_read(B(cache(**kw)), FAKE, 3, B(rows()), B(rows()), None) in (1, 2)
    assert msg in last()
    assert L().exl3_paged_attention(B(cache(**kw)), B(rows()), B(rows()), FAKE, FAKE, FAKE, 1, 1, 1, 3, 1.0, 0, None, 0,
                                    None) in (1, 2)
    assert msg in last()


def test_cache_write_and_read_refusals():
    c = cache()
    assert L().exl3_cache_write(B(c), B(rows(heads=3)), B(rows()), FAKE, 3, None) == 1 and "the cache 4" in last()
    assert L().exl3_cache_write(B(c), B(rows()), B(rows()), None, 3, None) == 1 and "slots is NULL" in last()
    assert L().exl3_cache_write(B(c), B(rows()), B(rows(data=None)), FAKE, 3, None) == 1 and "v is NULL" in last()
    assert L().exl3_cache_write(B(c), B(rows()), B(rows()), None, 0, None) == 0
    assert L().exl3_cache_read(B(c), FAKE, 3, B(rows(head=0)), B(rows()), None) == 1 and "overlap" in last()
    assert L().exl3_cache_read(B(c), FAKE, 3, B(rows()), B(rows(heads=2)), None) == 1 and "v_out 2" in last()
    assert L().exl3_cache_read(None, FAKE, 3, B(rows()), B(rows()), None) == 1 and "cache is NULL" in last()
    far = rows(data=FAKE + 4096 * 64)
    args = (FAKE, FAKE, 3, B(rows()), B(far), B(rows()), None, B(rows()), None)
    assert L().exl3_rope_cache_write(B(c), B(rotary(rot=8)), *args) == 1 and "rot=8" in last()
    assert L().exl3_rope_cache_write(B(c), B(rotary()), FAKE, None, 3, B(rows()), B(far), B(rows()), None, B(rows()),
                                     None) == 1 and "slots is NULL" in last()
    assert L().exl3_rope_cache_write(B(c), B(rotary()), FAKE, FAKE, 3, B(rows()), B(far), B(rows()), B(rows(token=1024)),
                                     B(rows()), None) == 1 and "k_out starts at its input" in last()


def paged(c=None, q=None, out=None, cu=FAKE, kv=FAKE, table=FAKE, stride=4, width=4, batch=2, tokens=3, scale=1.0, window=0,
          ws=None, n=0):
    return L().exl3_paged_attention(B(c or cache()), B(q or rows(8)), B(out or rows(8)), cu, kv, table, stride, width, batch,
                                    tokens, scale, window, ws, n, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(q=rows(6), out=rows(6)), "6 query heads must be a multiple of the 4"),
    (dict(out=rows(4)), "out has 4 heads, q 8"),
    (dict(batch=-1), "batch=-1"), (dict(batch=0), "batch=0 with 3 tokens"), (dict(batch=(1 << 16) + 1), "batch=65537"),
    (dict(width=-1), "page table width=-1"), (dict(window=-2), "window=-2"),
    (dict(scale=0.0), "scale=0"), (dict(scale=-1.0), "scale=-1"), (dict(scale=math.nan), "scale=nan"),
    (dict(scale=math.inf), "scale=inf"), (dict(cu=None), "cu_q is NULL"), (dict(kv=None), "kv_len is NULL"),
    (dict(table=None), "page_table is NULL"), (dict(table=FAKE + 1), "not 4-byte aligned"),
    (dict(out=rows(8, token=512)), "overlap"), (dict(tokens=-4), "tokens=-4"),
])
def test_paged_refusals(kw, msg):
    assert paged(**kw) in (1, 2)
    assert msg in last()


def test_paged_without_tokens():
    assert paged(tokens=0, batch=0, cu=None, kv=None, table=None) == 0


def prompt(q=None, k=None, v=None, out=None, cu=FAKE, batch=2, tokens=5, d=128, dtype=1, causal=1, window=0, scale=1.0):
    return L().exl3_prompt_attention(B(q or rows(8)), B(k or rows(2)), B(v or rows(2)), B(out or rows(8)), cu, batch, tokens,
                                     d, dtype, causal, window, scale, None, 0, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(k=rows(3)), "k has 3 heads, v 2"), (dict(k=rows(3), v=rows(3)), "multiple of the 3"),
    (dict(causal=2), "causal=2"), (dict(causal=0, window=4), "a window is causal"), (dict(window=-1), "window=-1"),
    (dict(d=32), "head_dim=32"), (dict(cu=None), "cu is NULL"), (dict(batch=0), "batch=0"), (dict(dtype=3), "dtype=3"),
    (dict(v=rows(2, data=FAKE + 2)), "v="), (dict(scale=0.0), "scale=0"),
])
def test_prompt_refusals(kw, msg):
    assert prompt(**kw) in (1, 2)
    assert msg in last()


def test_windows_and_strides_past_32_bit_offsets_are_refused():
    assert paged(window=(1 << 30) + 1) == 1 and "window=1073741825" in last()
    assert prompt(window=(1 << 30) + 1) == 1 and "window=1073741825" in last()
    wide = rows(2, token=(1 << 22) + 8)
    assert prompt(k=wide) == 2 and "token strides of k (4194312)" in last()
    assert prompt(v=wide) == 2 and "and v (4194312)" in last()


def test_workspace_holds_counters_and_parts_and_is_needed_only_with_few_tiles():
    """One token over one cache is split, so it needs the counters and partial sums; prompts whose tiles fill the
    GPU four times over need nothing; a call with a shorter workspace than it needs is refused."""
    need = ex.attention_workspace_bytes(1, 1, 32, 8, 128)
    assert need > 65536 and (need - 65536) % (16 * 130 * 4) == 0
    assert ex.attention_workspace_bytes(1, 100000, 32, 8, 128) == 0
    assert ex.attention_workspace_bytes(0, 0, 32, 8, 128) >= 0
    for short in (0, need - 16):
        st = paged(q=rows(32), out=rows(32), c=cache(heads=8, bits=16, page=16, k_page_bytes=8 * 16 * 256, v_page_bytes=8 * 16 * 256),
                   batch=1, tokens=1, ws=FAKE if short else None, n=short)
        assert st == 3 and f"short by {need - short}" in last()


def test_workspace_query_refusals():
    for args in ((-1, 1, 4, 4, 128), (1, -1, 4, 4, 128), (1, 1, 5, 4, 128), (1, 1, 4, 0, 128), (1, 1, 4, 4, 100)):
        with pytest.raises(ex.Exl3Error):
            ex.attention_workspace_bytes(*args)


# ------------------------------------------------------------ the binding

def test_binding_refuses_before_the_library():
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        at._rows(q, "q")
    with pytest.raises(ValueError, match=r"expected \[tokens, heads"):
        at._rows(torch.zeros(3, 4, 96), "q")
    with pytest.raises(ValueError, match=r"expected \[tokens, heads"):
        at._rows(torch.zeros(3, 128), "q")
    with pytest.raises(ValueError, match="float32"):
        ex.Rope(torch.zeros(3, 4, 2, dtype=torch.float64))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ex.Rope(torch.zeros(3, 8, 2))
    for bad in (dict(rotary_dim=20), dict(rotary_dim=0), dict(linear=0.0), dict(yarn=(0.5, 100))):
        with pytest.raises(ValueError):
            ex.Rope.make(**{**dict(rotary_dim=64, base=1e4, positions=4, device="cpu"), **bad})
    with pytest.raises(ValueError, match="qkv has shape"):
        ex.split_heads(torch.zeros(3, 100), 2, 1, 64)
    with pytest.raises(ValueError, match="dense int32"):
        at._ints(torch.zeros(3, dtype=torch.int64), "slots", 3, torch.device("cpu"))
    with pytest.raises(ValueError, match="dense int32"):
        at._ints(torch.zeros(4, dtype=torch.int32), "slots", 3, torch.device("cpu"))
    with pytest.raises(ValueError, match="expected bfloat16 or float16"):
        at._dtype_id(torch.float32, "q")


def test_binding_checks_the_cache_tensors():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    s = torch.zeros(4, 2, 16, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="needs k_scale"):
        ex.KvCache(k, k)
    with pytest.raises(ValueError, match="must be alike"):
        ex.KvCache(k, k[:2], s, s, torch.bfloat16)
    with pytest.raises(ValueError, match="do not match scales"):
        ex.KvCache(k, k, s[..., :3], s[..., :3], torch.bfloat16)
    with pytest.raises(ValueError, match="v_scale"):
        ex.KvCache(k, k, s, s[:3], torch.bfloat16)
    with pytest.raises(ValueError, match="no scales"):
        ex.KvCache(k.bfloat16(), k.bfloat16(), s, s)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ex.KvCache(k, k, s, s, torch.bfloat16)
    with pytest.raises(ValueError, match="bits=6"):
        ex.KvCache.empty(1, 16, 1, 64, 6)


def test_split_heads_are_views():
    qkv = torch.arange(2 * 8 * 64).reshape(2, 512)
    q, k, v = ex.split_heads(qkv, 4, 2, 64)
    assert q.shape == (2, 4, 64) and k.shape == v.shape == (2, 2, 64)
    assert torch.equal(torch.cat((q, k, v), 1).reshape(2, 512), qkv) and q.data_ptr() == qkv.data_ptr()


# -------------------------------------------- the reference the GPU tests use

def test_reference_rotation_against_complex_numbers():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 3, 64, generator=g).bfloat16()
    table = torch.randn(10, 16, 2, generator=g)
    pos = torch.tensor([0, 9, 3, 3, 7])
    z = torch.view_as_complex(table.double())[pos][:, None]
    y, bound = ref.rotate(x, table, pos, True)
    want = torch.view_as_real(torch.view_as_complex(x.double()[..., :32].reshape(5, 3, 16, 2)) * z).reshape(5, 3, 32)
    assert (y[..., :32] - want).abs().max() < 1e-12 and torch.equal(y[..., 32:], x.double()[..., 32:])
    y, _ = ref.rotate(x, table, pos, False)
    want = torch.complex(x.double()[..., :16], x.double()[..., 16:32]) * z
    assert (torch.cat((want.real, want.imag), -1) - y[..., :32]).abs().max() < 1e-12
    assert (bound[..., 32:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [8, 4])
def test_reference_quantiser(bits, dtype):
    """Against a search over every code at every scale, and torch's own e4m3."""
    g = torch.Generator().manual_seed(bits)
    x = (torch.randn(40, 32, generator=g) * torch.exp2(torch.randint(-12, 9, (40, 1), generator=g).float())).to(dtype)
    got = ref.quantise(x, bits)
    if bits == 8:
        codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        codes = codes[torch.isfinite(codes)]
    else:
        codes = torch.tensor(ref.E2M1 + tuple(-e for e in ref.E2M1)).double()
    lo, hi = ref.RANGE[(dtype, bits)]
    for row, out in zip(x.double(), got):
        e = lo
        while row.abs().max() > (448 if bits == 8 else 7) * 2.0 ** e and e < hi:
            e += 1
        gap = (row[:, None] - codes * 2.0 ** e).abs().amin(1)
        assert torch.allclose((row - out).abs(), gap, rtol=0, atol=0)
        if bits == 8:
            assert torch.equal(out, (row * 2.0 ** -e).float().to(torch.float8_e4m3fn).double() * 2.0 ** e)


def test_reference_attention_against_softmax():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, h, 64, generator=g).double() for n, h in ((6, 4), (11, 2), (11, 2)))
    seen = ref.mask(6, 11, True, 7)
    o, bound = ref.attend(q, k, v, seen, 0.125, torch.bfloat16)
    for h in range(4):
        w = (q[:, h] @ k[:, h // 2].T * 0.125).masked_fill(~seen, -math.inf)
        assert (torch.softmax(w, -1) @ v[:, h // 2] - o[:, h]).abs().max() < 1e-12
    # rounding to the type lies inside the bound, a dropped key outside
    assert ((o.bfloat16().double() - o).abs() <= bound).all()
    seen[:, 9] = False
    assert ((ref.attend(q, k, v, seen, 0.125, torch.bfloat16)[0] - o)[4:].abs() > bound[4:]).any()
