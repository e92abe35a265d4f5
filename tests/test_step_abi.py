"""The C ABI of include/exl3_step.h and its binding on the CPU: exports, the
header as C, and every refusal.  No call here reaches a kernel launch (there is
no GPU)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import linear_exl3_input_amd as ex
import step_reference as step
from linear_exl3_input_amd import attention as at
from test_attention_abi import FAKE, ROOT, cache, last, rotary, rows

pytestmark = pytest.mark.skipif(not os.path.exists(ex.lib_path()), reason="libexl3.so not built")

B = ctypes.byref


def L():
    return at._lib()


def test_exports_every_header_symbol():
    names = at.attn_header_symbols(at.STEP_HEADER)
    for name in ("exl3_norm_rope", "exl3_norm_rope_cache_write", "exl3_cache_extend"):
        assert name in names
    for name in names:
        assert hasattr(ex.load(), name), name
        assert getattr(L(), name).argtypes is not None, name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "exl3_step.h"\nint main(void) { exl3_rotary_axes r; exl3_head_norm n; r.axes = 1; n.eps = 1; '
                   'return r.axes - (int)n.eps; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-fsyntax-only", str(src)],
                   check=True)


# ------------------------------------------------------- norms and axes

def axes(n=3, words=(0x24924924,) * 8, **kw):
    return at._RotaryAxes(rotary(**kw), n, (ctypes.c_uint32 * 8)(*words))


def norm(q=FAKE, k=FAKE, q_rows=1, k_rows=1, eps=1e-6):
    return at._HeadNorm(q, k, q_rows, k_rows, eps)


def norm_rope(r=None, n=norm(), tokens=4, d=128, dtype=1, q=None, qo=None, k=None, ko=None, pos=FAKE, stride=4):
    ref = lambda x: None if x is None else B(x)  # noqa: E731
    return L().exl3_norm_rope(B(r or axes()), ref(n), pos, stride, tokens, d, dtype, B(q or rows()), B(qo or rows()), ref(k),
                              ref(ko), None)


def norm_write(c=None, r=None, n=norm(), tokens=4, q=None, qo=None, k=None, ko=None, v=None, pos=FAKE, slots=FAKE, stride=4):
    ref = lambda x: None if x is None else B(x)  # noqa: E731
    return L().exl3_norm_rope_cache_write(B(c or cache()), B(r or axes()), ref(n), pos, stride, slots, tokens, B(q or rows()),
                                          B(qo or rows()), B(k or rows()), ref(ko), B(v or rows()), None)


COMMON = [(dict(r=axes(0)), 1, "axes=0"), (dict(r=axes(5)), 1, "axes=5"), (dict(r=axes(2)), 1, "turns by axis 2 of 2"),
          (dict(r=axes(rot=24)), 1, "rot=24"), (dict(r=axes(rot=256)), 1, "rot=256"), (dict(r=axes(table=None)), 1, "rotary table is NULL"),
          (dict(r=axes(interleaved=2)), 1, "interleaved=2"), (dict(r=axes(positions=0)), 1, "0 positions"),
          (dict(stride=-1), 1, "axis_stride=-1"), (dict(stride=(1 << 40) + 1), 1, "axis_stride"), (dict(pos=None), 1, "positions is NULL"),
          (dict(n=norm(q=None)), 1, "norm q is NULL"), (dict(n=norm(q=FAKE + 4)), 1, "not 16-byte aligned"),
          (dict(n=norm(q_rows=2)), 1, "weights of 2 query heads, q has 4"), (dict(n=norm(q_rows=0)), 1, "weights of 0 query heads"),
          (dict(n=norm(k_rows=3), k=rows(), ko=rows()), 1, "weights of 3 key heads, k has 4"),
          (dict(n=norm(k=None), k=rows(), ko=rows()), 1, "norm k is NULL"), (dict(n=norm(eps=0.0)), 1, "eps=0"),
          (dict(n=norm(eps=-1.0)), 1, "eps=-1"), (dict(n=norm(eps=math.nan)), 1, "eps="), (dict(n=norm(eps=2.0)), 1, "eps=2"),
          (dict(tokens=-1), 1, "tokens=-1"), (dict(tokens=(1 << 20) + 1), 2, "exceeds the supported"),
          (dict(q=rows(data=None)), 1, "q is NULL"), (dict(qo=rows(head=64)), 1, "overlap"),
          (dict(qo=rows(heads=3)), 1, "q_out has 3 heads"), (dict(q=rows(head=100)), 1, "multiples of 8"),
          (dict(q=rows(token=1024)), 1, "starts at its input with other strides")]


@pytest.mark.parametrize("kw,status,msg", COMMON + [(dict(k=rows()), 1, "given together"), (dict(d=96), 2, "head_dim=96"),
                                                    (dict(dtype=3), 1, "dtype=3")])
def test_norm_rope_refusals(kw, status, msg):
    assert norm_rope(**kw) == status and msg in last(), last()


@pytest.mark.parametrize("kw,status,msg", COMMON + [(dict(slots=None), 1, "slots is NULL"), (dict(k=rows(3)), 1, "k has 3 heads"),
                                                    (dict(v=rows(5)), 1, "v 5"), (dict(c=cache(bits=5)), 1, "bits=5")])
def test_norm_write_refusals(kw, status, msg):
    assert norm_write(**kw) == status and msg in last(), last()


def test_axes_past_the_rotated_pairs_do_not_matter():
    words = [0x24924924, 0x24924924] + [0xFFFFFFFF] * 6  # 32 pairs of axes 0..2
    assert norm_rope(r=axes(3, words), tokens=0) == 0
    assert norm_rope(r=axes(3, words, rot=80), tokens=0) == 1 and "pair 32 turns by axis 3 of 3" in last()


def test_without_tokens_no_pointers_are_needed():
    assert norm_rope(tokens=0, pos=None, q=rows(data=None), qo=rows(data=None)) == 0
    assert norm_write(tokens=0, pos=None, slots=None) == 0


# --------------------------------------------------------------- tables

def ints(n=0):
    return FAKE + 0x10000 * n


def extend(pages=10, page=16, q=ints(1), kv=ints(2), batch=3, table=ints(3), stride=4, width=4, free=ints(4), n_free=5, taken=None,
           tokens=6, cu=ints(5), out=ints(6), pos=ints(7), slots=ints(8), counts=ints(9)):
    return L().exl3_cache_extend(pages, page, q, kv, batch, table, stride, width, free, n_free, taken, tokens, cu, out, pos, slots,
                                 counts, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(page=24), "page_size=24"), (dict(page=8), "page_size=8"), (dict(pages=0), "0 pages"), (dict(pages=1 << 28), "pages of 16"),
    (dict(batch=-1), "batch=-1"), (dict(batch=65537), "batch=65537"), (dict(tokens=-1), "tokens=-1"),
    (dict(tokens=(1 << 20) + 1), "tokens="), (dict(n_free=-1), "n_free=-1"), (dict(width=-1), "width=-1"), (dict(stride=3), "overlap"),
    (dict(stride=-4, batch=1), "stride=-4"), (dict(stride=(1 << 40) + 1), "2^40"), (dict(q=None), "q_len is NULL"),
    (dict(kv=None), "kv_len is NULL"), (dict(table=None), "page_table is NULL"), (dict(free=None), "free_pages is NULL"),
    (dict(taken=3), "taken=0x3 is not 4-byte aligned"), (dict(cu=None), "cu_q is NULL"), (dict(out=None), "kv_out is NULL"),
    (dict(pos=None), "positions is NULL"), (dict(slots=None), "slots is NULL"), (dict(counts=None), "counts is NULL"),
    (dict(slots=ints(8) + 2), "not 4-byte aligned"), (dict(out=ints(2)), "kv_len and kv_out overlap"),
    (dict(out=ints(2) + 8), "kv_len and kv_out overlap"), (dict(cu=ints(1) - 12), "q_len and cu_q overlap"),
    (dict(table=ints(2) - 44), "kv_len and page_table overlap"), (dict(free=ints(3) + 40), "free_pages and page_table overlap"),
    (dict(taken=ints(9) + 4), "taken and counts overlap"), (dict(pos=ints(8) - 20), "positions and slots overlap")])
def test_extend_refusals(kw, msg):
    assert extend(**kw) == 1 and msg in last(), last()


# ----------------------------------------------------------- the binding

def test_binding_refuses_before_the_library():
    table = torch.zeros(4, 16, 2)
    for bad in ([0] * 15, [0] * 17, [0] * 15 + [4], [-1] + [0] * 15):
        with pytest.raises(ValueError, match="must name an axis"):
            at._axes(bad, 32)
    for bad in ((16,) * 2, (4, 4, 4, 2, 2), (8, 8, 0), (), (20, -4)):
        with pytest.raises(ValueError, match="sections"):
            ex.Rope.make(32, 1e4, 4, device="cpu", sections=bad)
    assert at._axes(None, 32)[:2] == (None, 1) and at._axes([0] * 16, 32)[1] == 1 and at._axes([3] * 128, 256)[2][7] == 2 ** 32 - 1
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ex.Rope(table, axes=[0] * 16)
    w = torch.ones(128)
    for kw, msg in ((dict(q_weight=torch.ones(100)), "expected floating"), (dict(q_weight=torch.ones(128, dtype=torch.int32)), "expected floating"),
                    (dict(q_weight=torch.ones(2, 2, 128)), "expected floating"), (dict(q_weight=torch.ones(0, 128)), "expected floating"),
                    (dict(q_weight=w), "must be a GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            ex.HeadNorm(**kw)
    with pytest.raises(ValueError, match="page_table must be int32"):
        at._page_table(torch.zeros(3, 4, dtype=torch.int64), 3, torch.device("cpu"))
    with pytest.raises(ValueError, match="page_table must be int32"):
        at._page_table(torch.zeros(4, 3, dtype=torch.int32).T, 3, torch.device("cpu"))


# ------------------------------------------- the reference against others

def test_reference_norm_against_torch():
    x, w = torch.randn(5, 3, 64, dtype=torch.float64), torch.rand(64, dtype=torch.float64)
    want = torch.nn.functional.rms_norm(x, (64,), w, 1e-5)
    assert (step.normed(x, w, 1e-5)[0] - want).abs().max() < 1e-12


def test_reference_axes_against_complex_numbers():
    r = torch.randn(7, 8, dtype=torch.float64)
    table = torch.stack((r.cos(), r.sin()), -1)
    x = torch.randn(5, 3, 24, dtype=torch.float64)
    pos, axes_ = torch.randint(0, 7, (3, 5)), [0, 2, 1, 1, 0, 2, 2, 1]
    angle = torch.stack([r[pos[a], i] for i, a in enumerate(axes_)], 1)[:, None]
    for inter in (False, True):
        y, _ = step.turned(x, torch.zeros_like(x), table, pos, axes_, inter, torch.bfloat16)
        a, b = (x[..., 0:16:2], x[..., 1:16:2]) if inter else (x[..., :8], x[..., 8:16])
        z = torch.complex(a, b) * torch.polar(torch.ones_like(angle), angle)
        got = torch.complex(y[..., 0:16:2], y[..., 1:16:2]) if inter else torch.complex(y[..., :8], y[..., 8:16])
        assert (got - z).abs().max() < 1e-12 and torch.equal(y[..., 16:], x[..., 16:])


def test_reference_tables_by_hand():
    got = step.extended(10, 16, [3, 0, 20], [14, 16, 0], [[4, -1], [5, -1], [-1, -1]], [7, 8, 9], 26)
    assert got[0] == [0, 3, 3, 23] and got[1] == [17, 16, 20] and got[4] == [23, 3]
    assert got[2] == [14, 15, 16, *range(20), 0, 0, 0]
    assert got[3] == [4 * 16 + 14, 4 * 16 + 15, 7 * 16, *range(128, 144), *range(144, 148), -1, -1, -1]
    assert got[5] == [[4, 7], [5, -1], [8, 9]]


# ------------------------------------------------- windows with first tokens

def paged_sinks(window=5, sinks=4, tokens=3, ws=None, n=0, **kw):
    a = dict(c=cache(), q=rows(), out=rows(), cu=FAKE, kv=FAKE, table=FAKE, stride=4, width=4, batch=2, scale=1.0)
    a.update(kw)
    return L().exl3_paged_attention_sinks(B(a["c"]), B(a["q"]), B(a["out"]), a["cu"], a["kv"], a["table"], a["stride"], a["width"],
                                          a["batch"], tokens, a["scale"], window, sinks, ws, n, None)


def prompt_sinks(window=5, sinks=4, tokens=5, **kw):
    a = dict(q=rows(), k=rows(), v=rows(), out=rows(), cu=FAKE, batch=2, d=128, dtype=1, scale=1.0)
    a.update(kw)
    return L().exl3_prompt_attention_sinks(B(a["q"]), B(a["k"]), B(a["v"]), B(a["out"]), a["cu"], a["batch"], tokens, a["d"],
                                           a["dtype"], window, sinks, a["scale"], None, 0, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(window=0), "window=0"), (dict(window=-1), "window=-1"), (dict(window=(1 << 30) + 1), "window="),
    (dict(sinks=-1), "sinks=-1"), (dict(sinks=(1 << 20) + 1), "sinks=1048577"), (dict(cu=None), "cu"), (dict(batch=0), "batch=0"),
    (dict(scale=0.0), "scale=0"), (dict(out=rows(3)), "out has 3 heads"), (dict(q=rows(6), out=rows(6)), "multiple of the 4")])
def test_sinks_refusals(kw, msg):
    assert paged_sinks(**kw) == 1 and msg in last(), last()
    assert prompt_sinks(**kw) == 1 and msg in last(), last()


def test_sinks_need_the_workspace_that_the_plain_calls_need():
    need = ex.attention_workspace_bytes(2, 3, 4, 4, 128)
    assert need > 0 and paged_sinks() == 3 and f"needs {need}" in last()
    assert paged_sinks(tokens=0) == 0 and prompt_sinks(tokens=0) == 0


# ------------------------------------------------------- shared prefixes

def prefix(tokens=3, groups=1, group_cu=FAKE, lens=FAKE, ws=None, n=0, **kw):
    a = dict(c=cache(), q=rows(), out=rows(), cu=FAKE, kv=FAKE, table=FAKE, stride=4, width=4, batch=2, scale=1.0)
    a.update(kw)
    return L().exl3_prefix_attention(B(a["c"]), B(a["q"]), B(a["out"]), a["cu"], a["kv"], a["table"], a["stride"], a["width"],
                                     a["batch"], tokens, group_cu, lens, groups, a["scale"], ws, n, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(groups=-1), "groups=-1"), (dict(groups=3), "groups=3, must be 0..batch=2"), (dict(group_cu=None), "group_cu is NULL"),
    (dict(lens=None), "prefix_len is NULL"), (dict(lens=FAKE + 2), "not 4-byte aligned"), (dict(cu=None), "cu"), (dict(batch=0), "batch=0"),
    (dict(scale=-1.0), "scale=-1"), (dict(out=rows(3)), "out has 3 heads"), (dict(q=rows(6), out=rows(6)), "multiple of the 4"),
    (dict(kv=None), "kv_len is NULL"), (dict(stride=-4), "negative")])
def test_prefix_refusals(kw, msg):
    assert prefix(**kw) == 1 and msg in last(), last()


def test_prefix_workspace():
    need = ex.prefix_attention_workspace_bytes(2, 3, 1, 4, 4, 128)
    state = 3 * 4 * 132 * 4
    assert need >= ex.attention_workspace_bytes(2, 3, 4, 4, 128) + state and need >= ex.attention_workspace_bytes(1, 3, 4, 4, 128) + state
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE, 0)):
        assert prefix(ws=ws, n=n) == 3 and f"needs {need}" in last()
    assert prefix(ws=FAKE + 4, n=need) == 1 and "not 16-byte aligned" in last()
    assert prefix(tokens=0) == 0 and prefix(tokens=0, groups=0, group_cu=None, lens=None) == 0
    for args in ((-1, 1, 0, 4, 4, 128), (1, 1, 2, 4, 4, 128), (1, 1, -1, 4, 4, 128), (1, 1, 1, 5, 4, 128), (1, 1, 1, 4, 4, 100)):
        with pytest.raises(ex.Exl3Error):
            ex.prefix_attention_workspace_bytes(*args)


def test_the_prefix_workspace_is_bounded():
    """At most 1 GiB more than the groups' arrays (24 bytes a sequence and a group) and parts of own keys, whatever the sizes."""
    for d in (64, 128, 256):
        for hq, hkv in ((1, 1), (32, 8), (64, 8), (24, 4), (1024, 1024), (1024, 8)):
            for batch in (1, 16, 256, 2048, 16384, 65536):
                for each in (1, 8, 64, 512):
                    if batch * each <= 1 << 20:
                        for groups in {0, 1, batch // 8, batch}:
                            need = ex.prefix_attention_workspace_bytes(batch, batch * each, groups, hq, hkv, d)
                            plain = ex.attention_workspace_bytes(batch, batch * each, hq, hkv, d)
                            assert need <= (1 << 30) + (1 << 20) + plain + 48 * batch + 16384 * 16 * (d + 2) * 4, (batch, each, groups, hq, hkv, d)
