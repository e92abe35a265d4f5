"""What stands between a decoder's q/k/v and output projections on an MI355X:
rotary positions (with norms of the heads, over several axes), a paged key/value
cache that is quantized as it is written, its page tables and slots from the
requests' lengths, attention over that cache (of sequences that share a prefix
too) and attention over packed prompts.

A ctypes binding over ``include/exl3_attn.h`` and ``include/exl3_step.h`` like
the package's own: tensor metadata is checked here, everything else by the
library, and there is no fallback.  One decoder layer's step of a server:

    rope = Rope.make(rotary_dim, base=1e6, positions=32768)
    norm = HeadNorm(q_weight, k_weight)
    cache = KvCache.empty(pages, page_size, kv_heads, head_dim, bits=8)
    ...
    step = cache_extend(cache, q_len, kv_len, page_table, free_pages, tokens)
    ...
    qkv = forward(w_qkv, x)                       # [tokens, (hq + 2*hkv)*d]
    q, k, v = split_heads(qkv, hq, hkv, head_dim)      # views
    q = rope_cache_write(cache, rope, step.positions, step.slots, q, k, v, norm=norm)
    y = paged_attention(cache, q, step.cu_q, step.kv_len, page_table)
    x = forward(w_o, y.view(tokens, -1))

Rows may have any token and head stride (a multiple of 8 values), so the
views of a fused projection's output are taken as they are.  positions,
slots, lengths and page tables are int32 tensors on the GPU; nothing here
reads them back, so every call may be captured in a graph.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _BF16, _F16, _HERE, _check, _workspace, _workspaces, _ws_needs_zero, load

__all__ = ["Rope", "KvCache", "split_heads", "rope", "cache_write", "cache_read", "rope_cache_write",
           "paged_attention", "prompt_attention", "attention_workspace_bytes", "HeadNorm", "CacheStep", "cache_extend",
           "prefix_attention", "prefix_attention_workspace_bytes"]

ATTN_HEADER = os.path.join(os.path.dirname(_HERE), "include", "exl3_attn.h")
STEP_HEADER = os.path.join(os.path.dirname(_HERE), "include", "exl3_step.h")
HEAD_DIMS = (64, 128, 256)


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class _Rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _RotaryAxes(ctypes.Structure):
    _fields_ = [("rotary", _Rotary), ("axes", ctypes.c_int32), ("axis_of", ctypes.c_uint32 * 8)]


class _HeadNorm(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_rows", ctypes.c_int32), ("k_rows", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_page_bytes", ctypes.c_int64), ("v_page_bytes", ctypes.c_int64),
                ("k_scale_page_bytes", ctypes.c_int64), ("v_scale_page_bytes", ctypes.c_int64),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("bits", ctypes.c_int32)]


_fns = None


def _lib():
    global _fns
    if _fns is None:
        L = load()
        vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        R, T, C = ctypes.POINTER(_Rows), ctypes.POINTER(_Rotary), ctypes.POINTER(_Cache)
        A, N = ctypes.POINTER(_RotaryAxes), ctypes.POINTER(_HeadNorm)
        sig = {
            "exl3_rope": (i32, [T, vp, i32, i32, i32, R, R, R, R, vp]),
            "exl3_cache_write": (i32, [C, R, R, vp, i32, vp]),
            "exl3_rope_cache_write": (i32, [C, T, vp, vp, i32, R, R, R, R, R, vp]),
            "exl3_cache_read": (i32, [C, vp, i32, R, R, vp]),
            "exl3_paged_attention": (i32, [C, R, R, vp, vp, vp, i64, i32, i32, i32, f32, i32, vp, sz, vp]),
            "exl3_prompt_attention": (i32, [R, R, R, R, vp, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]),
            "exl3_attention_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
            "exl3_norm_rope": (i32, [A, N, vp, i64, i32, i32, i32, R, R, R, R, vp]),
            "exl3_norm_rope_cache_write": (i32, [C, A, N, vp, i64, vp, i32, R, R, R, R, R, vp]),
            "exl3_paged_attention_sinks": (i32, [C, R, R, vp, vp, vp, i64, i32, i32, i32, f32, i32, i32, vp, sz, vp]),
            "exl3_prompt_attention_sinks": (i32, [R, R, R, R, vp, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]),
            "exl3_prefix_attention": (i32, [C, R, R, vp, vp, vp, i64, i32, i32, i32, vp, vp, i32, f32, vp, sz, vp]),
            "exl3_prefix_attention_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32]),
            "exl3_cache_extend": (i32, [i32, i32, vp, vp, i32, vp, i64, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _fns = L
    return _fns


def attn_header_symbols(header: str = ATTN_HEADER) -> Tuple[str, ...]:
    """Every function that exl3_attn.h (or another header) declares."""
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    return tuple(sorted(set(re.findall(r"\b(exl3_[a-z_]+)\s*\(", text))))


_DTYPES = {torch.bfloat16: _BF16, torch.float16: _F16}


def _dtype_id(dtype: torch.dtype, name: str) -> int:
    i = _DTYPES.get(dtype)
    if i is None:
        raise ValueError(f"{name} has dtype {dtype}, expected bfloat16 or float16")
    return i


# A call of a few microseconds on the GPU should not take three times as long
# here: the current stream's handle straight from torch's binding (0.1 us; by
# way of a Stream object 2.7 us), outputs by empty_like (1.0 us; torch.empty
# with a shape, dtype and device 2.0 us), the workspace's lock only when there
# is something to do.
_raw_stream = torch._C._cuda_getCurrentRawStream
# The library launches on the current device and plans for it: a call whose
# tensors are on another one makes that current first.
_current_device = torch._C._cuda_getDevice


def _scratch(nbytes: int, device: torch.device, stream: int) -> Tuple[Optional[int], int]:
    if nbytes == 0:
        return None, 0
    key = (device.index, stream)
    ws = _workspaces.get(key)
    if ws is not None and ws.numel() >= nbytes and key not in _ws_needs_zero:
        return ws.data_ptr(), ws.numel()
    return _workspace(nbytes, device)


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> _Rows:
    """The view of a [tokens, heads, head_dim] tensor, checked against `like`'s tokens, dtype and device."""
    shape = t.shape
    if len(shape) != 3 or shape[2] not in HEAD_DIMS:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens, heads, 64, 128 or 256]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if like is not None and like is not t:
        if t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
        if shape[0] != like.shape[0] or shape[2] != like.shape[2]:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {like.shape[0]} tokens of "
                             f"{like.shape[2]}-value heads")
    tokens, heads, last = t.stride()
    if last != 1:
        raise ValueError(f"{name} has stride {last} in its last dimension, expected 1")
    # the stride of a dimension of one is never used and may be anything
    return _Rows(t.data_ptr(), tokens if shape[0] > 1 else 0, heads if shape[1] > 1 else 0, shape[1])


def _ints(t: torch.Tensor, name: str, n: int, device) -> int:
    if t.dtype != torch.int32 or t.device != device or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a dense int32 tensor [{n}] on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    return t.data_ptr()


def _out(out: Optional[torch.Tensor], like: torch.Tensor, name: str) -> Tuple[torch.Tensor, _Rows]:
    """`out`, or a new dense tensor like the (checked) `like`, and its view."""
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        tokens, heads, dim = like.shape  # (strides as _rows gives them)
        return out, _Rows(out.data_ptr(), heads * dim if tokens > 1 else 0, dim if heads > 1 else 0, heads)
    if out.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {tuple(like.shape)}")
    return out, _rows(out, name, like)


def _window(window: int) -> int:
    """window for the library, which would take a number past 32 bits for what is left of it."""
    if not 0 <= window <= 1 << 30:
        raise ValueError(f"window={window}, must be 0 (none) to {1 << 30}")
    return window


def _sinks(sinks: int, window: int) -> int:
    """sinks for the library; 0 where nothing hides the first tokens anyway."""
    if not 0 <= sinks <= 1 << 20:
        raise ValueError(f"sinks={sinks}, must be 0 (none) to {1 << 20}")
    return sinks if window > 0 else 0


def _same_device(r: "Rope", q: torch.Tensor) -> None:
    if r.device != q.device:
        raise ValueError(f"the rotations are on {r.device}, q on {q.device}")


def split_heads(qkv: torch.Tensor, q_heads: int, kv_heads: int, head_dim: int):
    """q, k and v as views [tokens, heads, head_dim] of a fused projection's output [tokens, (q + 2 kv) * head_dim]."""
    if qkv.dim() != 2 or qkv.shape[1] != (q_heads + 2 * kv_heads) * head_dim:
        raise ValueError(f"qkv has shape {tuple(qkv.shape)}, expected [tokens, {(q_heads + 2 * kv_heads) * head_dim}]")
    x = qkv.unflatten(1, (q_heads + 2 * kv_heads, head_dim))
    return x[:, :q_heads], x[:, q_heads:q_heads + kv_heads], x[:, q_heads + kv_heads:]


class Rope:
    """A table of rotations, float32 [positions, rotary_dim/2, 2] (cosine, sine).

    interleaved False pairs value i with i + rotary_dim/2, True 2i with 2i + 1;
    values from rotary_dim on stay as they are.

    axes: the axis (0..3) whose position turns each pair, for tokens that have several (time, height
    and width of a video's patches); positions are then int32 [number of axes, tokens].  None: one axis,
    positions [tokens]."""

    def __init__(self, table: torch.Tensor, interleaved: bool = False, axes: Optional[Sequence[int]] = None):
        if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32 or not table.is_contiguous():
            raise ValueError("table must be a contiguous float32 tensor [positions, rotary_dim/2, 2]")
        if not table.is_cuda:
            raise ValueError("table must be a GPU tensor")
        self.table, self.interleaved, self.device = table, bool(interleaved), table.device
        self.positions, self.rotary_dim = table.shape[0], 2 * table.shape[1]
        self._view = _Rotary(table.data_ptr(), self.positions, self.rotary_dim, int(self.interleaved))
        self._ref = ctypes.byref(self._view)
        self.axes, self.n_axes, words = _axes(axes, self.rotary_dim)
        self._axes_view = _RotaryAxes(self._view, self.n_axes, words)
        self._axes_ref = ctypes.byref(self._axes_view)

    @classmethod
    def make(cls, rotary_dim: int, base: float, positions: int, interleaved: bool = False, linear: float = 1.0,
             ntk: float = 1.0, yarn: Optional[Tuple[float, int]] = None, yarn_turns: Tuple[float, float] = (1.0, 32.0),
             yarn_gain: Optional[float] = None, yarn_ramp: str = "pairs", device="cuda",
             sections: Optional[Sequence[int]] = None, in_turn: bool = False) -> "Rope":
        """Frequencies base^(-2i/rotary_dim), stretched for contexts longer than trained:

        linear f: every position is divided by f.
        ntk f: the base becomes base * f^(rotary_dim / (rotary_dim - 2)), so the slowest pair slows by f
            and the fastest stays.
        yarn (f, n): pairs that turn fewer than yarn_turns[0] times in the n trained positions slow by f,
            those that turn more than yarn_turns[1] times stay; cosines and sines are multiplied by yarn_gain
            (default 0.1 ln f + 1).  Between them is a ramp, and a model needs the one it was trained with:
            yarn_ramp "pairs": linear in the pair's index, from the last pair that turns yarn_turns[1] times
                to the first that turns yarn_turns[0] times or fewer (as released YaRN models have it);
            yarn_ramp "turns": linear in the number of turns (with yarn_turns=(1, 4), yarn_gain=1 the
                smoothing between a low and a high frequency factor of 1 and 4).

        sections: the pairs that each of several axes turns, rotary_dim/2 in all: the first sections[0] pairs by
        axis 0, the next sections[1] by axis 1 and so on; in_turn: pair i by axis i % len(sections) as long as that
        axis has pairs left, and by axis 0 after that.

        The angles are computed in float64 and the cosines and sines rounded to float32."""
        axes = None if sections is None else _axes_of_sections(sections, rotary_dim, in_turn)
        inv, gain = _frequencies(rotary_dim, base, linear, ntk, yarn, yarn_turns, yarn_gain, yarn_ramp)
        if positions < 1:
            raise ValueError(f"positions={positions} must be at least 1")
        a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv.to(device)
        return cls((torch.stack((a.cos(), a.sin()), -1) * gain).float(), interleaved, axes)


def _axes(axes: Optional[Sequence[int]], rotary_dim: int):
    """(axes, their number, two bits a pair for the library)."""
    words = (ctypes.c_uint32 * 8)()
    if axes is None:
        return None, 1, words
    axes = tuple(int(a) for a in axes)
    if len(axes) != rotary_dim // 2 or not all(0 <= a <= 3 for a in axes):
        raise ValueError(f"axes={axes} must name an axis 0..3 for each of {rotary_dim // 2} pairs")
    for i, a in enumerate(axes[:128]):
        words[i // 16] |= a << 2 * (i % 16)
    return axes, max(axes) + 1, words


def _axes_of_sections(sections: Sequence[int], rotary_dim: int, in_turn: bool) -> Tuple[int, ...]:
    n = len(sections)
    if not 1 <= n <= 4 or min(sections) < 1 or sum(sections) != rotary_dim // 2:
        raise ValueError(f"sections={tuple(sections)} must be 1 to 4 numbers of pairs, {rotary_dim // 2} in all")
    if in_turn:
        return tuple(i % n if i // n < sections[i % n] else 0 for i in range(rotary_dim // 2))
    return tuple(a for a, pairs in enumerate(sections) for _ in range(pairs))


def _frequencies(rotary_dim: int, base: float, linear: float, ntk: float, yarn: Optional[Tuple[float, int]],
                 yarn_turns: Tuple[float, float], yarn_gain: Optional[float], yarn_ramp: str) -> Tuple[torch.Tensor, float]:
    """The angle per position of each pair (float64 [rotary_dim/2]) and the gain of Rope.make."""
    if rotary_dim % 16 or rotary_dim < 16:
        raise ValueError(f"rotary_dim={rotary_dim} must be a multiple of 16")
    if not base > 1:
        raise ValueError(f"base={base} must be more than 1")
    if not (linear > 0 and ntk > 0) or (yarn is not None and not (yarn[0] >= 1 and yarn[1] >= 1)):
        raise ValueError(f"linear={linear}, ntk={ntk} must be positive, yarn={yarn} at least (1, 1)")
    if not 0 < yarn_turns[0] < yarn_turns[1]:
        raise ValueError(f"yarn_turns={yarn_turns} must be positive and rising")
    if yarn_ramp not in ("pairs", "turns"):
        raise ValueError(f'yarn_ramp={yarn_ramp!r} must be "pairs" or "turns"')
    if ntk != 1.0:
        base = base * ntk ** (rotary_dim / (rotary_dim - 2))
    half = rotary_dim // 2
    pair = torch.arange(half, dtype=torch.float64)
    inv = float(base) ** -(pair / half) / linear
    if yarn is None:
        return inv, 1.0
    factor, trained = yarn
    low, high = yarn_turns
    if yarn_ramp == "turns":
        keep = ((trained * inv / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    else:
        def pair_of(turns):  # where, as a real number, a pair would turn that often
            return half * math.log(trained / linear / (2 * math.pi * turns)) / math.log(base)

        first, last = max(math.floor(pair_of(high)), 0), min(math.ceil(pair_of(low)), rotary_dim - 1)
        keep = 1 - ((pair - first) / (last - first if last != first else 0.001)).clamp(0, 1)
    gain = yarn_gain if yarn_gain is not None else 0.1 * math.log(factor) + 1.0
    return inv * (keep + (1 - keep) / factor), gain


class HeadNorm:
    """Norms of each query and key head before the rotation: x / sqrt(mean(x^2) + eps) * weight over the head's
    values, in float32 up to the rounding after the rotation.

    q_weight, k_weight [head_dim], or [heads, head_dim] for weights of each head's own; copied as float32, plus one
    with one_plus (weights that are kept as their distance from one).  k_weight None: only q is given to the calls."""

    def __init__(self, q_weight: torch.Tensor, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 one_plus: bool = False):
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is None:
                continue
            if w.dim() not in (1, 2) or w.shape[-1] not in HEAD_DIMS or w.shape[0] == 0 or not w.is_floating_point():
                raise ValueError(f"{name} is {w.dtype} {tuple(w.shape)}, expected floating [64, 128 or 256] or "
                                 "[heads, 64, 128 or 256]")
            if not w.is_cuda:
                raise ValueError(f"{name} must be a GPU tensor")
            if w.device != q_weight.device or w.shape[-1] != q_weight.shape[-1]:
                raise ValueError(f"{name} is {tuple(w.shape)} on {w.device}, q_weight {tuple(q_weight.shape)} on "
                                 f"{q_weight.device}")
        if not 1e-30 <= eps <= 1:
            raise ValueError(f"eps={eps} must be 1e-30..1")
        self.eps, self.head_dim, self.device = float(eps), q_weight.shape[-1], q_weight.device
        # (a copy always: the caller may write to its tensors)
        self.q_weight, self.k_weight = (None if w is None else (w.detach().float() + (1.0 if one_plus else 0.0)).contiguous()
                                        for w in (q_weight, k_weight))
        rows = lambda w: 0 if w is None else 1 if w.dim() == 1 else w.shape[0]  # noqa: E731
        self._view = _HeadNorm(self.q_weight.data_ptr(), None if k_weight is None else self.k_weight.data_ptr(),
                               rows(q_weight), rows(k_weight), self.eps)
        self._ref = ctypes.byref(self._view)


class KvCache:
    """A paged cache of keys and values over tensors of the caller's.

    k, v [pages, heads, page_size, head_dim] of bfloat16 or float16 (16 bits), or
    uint8 codes [.., head_dim] (8 bits: e4m3) or [.., head_dim/2] (4 bits: e2m1, two
    in a byte, the even index in the low half) with uint8 scales [.., head_dim/32] and
    `dtype`, the type the values are read as.  Pages may be strided, e.g. one layer's
    slice of a tensor for all layers; within a page everything is dense."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None):
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError(f"k {k.dtype} {tuple(k.shape)} and v {v.dtype} {tuple(v.shape)} must be alike, "
                             "[pages, heads, page_size, ...]")
        pages, heads, page_size, last = k.shape
        if k.dtype == torch.uint8:
            if k_scale is None or v_scale is None or dtype is None:
                raise ValueError("a cache of codes needs k_scale, v_scale and dtype")
            head_dim = 32 * k_scale.shape[-1]
            bits = 8 * last // head_dim
            if bits not in (4, 8) or last * 8 != bits * head_dim:
                raise ValueError(f"codes of {last} bytes do not match scales of {k_scale.shape[-1]} blocks")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t.dtype != torch.uint8 or t.device != k.device or t.shape != (pages, heads, page_size, head_dim // 32):
                    raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected uint8 "
                                     f"{(pages, heads, page_size, head_dim // 32)} on {k.device}")
        else:
            if k_scale is not None or v_scale is not None or dtype not in (None, k.dtype):
                raise ValueError("a 16-bit cache has no scales and its tensors' own dtype")
            head_dim, bits, dtype = last, 16, k.dtype
        if not k.is_cuda:
            raise ValueError("k must be a GPU tensor")
        for t in (k, v) + ((k_scale, v_scale) if bits < 16 else ()):
            if not t[0].is_contiguous():
                raise ValueError(f"a page must be dense: strides {t.stride()} of shape {tuple(t.shape)}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, page_size, head_dim
        self.bits, self.dtype, self.device = bits, dtype, k.device
        def page_bytes(t):  # the stride of a single page is never used and may be anything
            return (t.stride(0) if pages > 1 else t[0].numel()) * t.element_size()

        scaled = bits < 16
        self._view = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if scaled else None,
                            v_scale.data_ptr() if scaled else None, page_bytes(k), page_bytes(v),
                            page_bytes(k_scale) if scaled else 0, page_bytes(v_scale) if scaled else 0, pages,
                            page_size, heads, head_dim, _dtype_id(dtype, "cache"), bits)
        self._ref = ctypes.byref(self._view)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, bits: int = 16,
              dtype: torch.dtype = torch.bfloat16, device="cuda") -> "KvCache":
        """A cache over new tensors (not initialized: slots that were not written hold anything)."""
        if bits not in (16, 8, 4):
            raise ValueError(f"bits={bits}, must be 16, 8 or 4")
        shape = (pages, heads, page_size)
        if bits == 16:
            k, v = (torch.empty((*shape, head_dim), dtype=dtype, device=device) for _ in range(2))
            return cls(k, v)
        k, v = (torch.empty((*shape, head_dim * bits // 8), dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.empty((*shape, head_dim // 32), dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, ks, vs, dtype)

    def slots(self, page_table: torch.Tensor, seq: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        """The int32 slots of tokens at `positions` of the sequences `seq` (rows of the page table); -1 where there is
        none: a hole of the table, or a position or sequence outside it (padding rows)."""
        rows, width = page_table.shape
        if rows == 0 or width == 0:
            return torch.full_like(positions, -1, dtype=torch.int32)
        at = positions // self.page_size
        s, i = seq.clamp(0, rows - 1), at.clamp(0, width - 1)
        page = page_table[s, i]
        missing = (s != seq) | (i != at) | (page.clamp(0, self.pages - 1) != page)
        slot = torch.add(positions % self.page_size, page, alpha=self.page_size)
        return torch.where(missing, -1, slot).int()


def _positions(r: Rope, positions: torch.Tensor, tokens: int, device) -> Tuple[int, int]:
    """The address and the axes' stride of positions [tokens], or [axes, tokens] for rotations of several axes."""
    if r.axes is None:
        return _ints(positions, "positions", tokens, device), 0
    if (positions.dtype != torch.int32 or positions.device != device or positions.dim() != 2 or
            positions.shape[0] != r.n_axes or positions.shape[1] != tokens or (tokens > 1 and positions.stride(1) != 1)):
        raise ValueError(f"positions must be int32 [{r.n_axes}, {tokens}] with dense rows on {device}, got "
                         f"{positions.dtype} {tuple(positions.shape)} on {positions.device}")
    return positions.data_ptr(), positions.stride(0) if r.n_axes > 1 else 0


def _norm(norm: Optional[HeadNorm], q: torch.Tensor):
    if norm is None:
        return None
    if norm.device != q.device or norm.head_dim != q.shape[2]:
        raise ValueError(f"the norms are of {norm.head_dim}-value heads on {norm.device}, q has {q.shape[2]} on {q.device}")
    return norm._ref


def rope(r: Rope, positions: torch.Tensor, q: torch.Tensor, k: Optional[torch.Tensor] = None,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, norm: Optional[HeadNorm] = None):
    """Rotates q [tokens, heads, head_dim] (and k) by their positions in one launch; returns q_out, or (q_out, k_out).
    An output may be its input (in place).  norm: the heads are normed first, in the same pass."""
    T, _, D = q.shape
    qr = _rows(q, "q")
    _same_device(r, q)
    if _current_device() != q.device.index:
        with torch.cuda.device(q.device):
            return rope(r, positions, q, k, q_out, k_out, norm)
    q_out, qo = _out(q_out, q, "q_out")
    kr = ko = None
    if k is not None:
        kr = ctypes.byref(_rows(k, "k", q))
        k_out, ko = _out(k_out, k, "k_out")
        ko = ctypes.byref(ko)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if norm is not None or r.axes is not None:
        at, stride = _positions(r, positions, T, q.device)
        _check(_lib().exl3_norm_rope(r._axes_ref, _norm(norm, q), at, stride, T, D, _dtype_id(q.dtype, "q"),
                                     ctypes.byref(qr), ctypes.byref(qo), kr, ko, _raw_stream(q.device.index)))
        return q_out if k is None else (q_out, k_out)
    _check(_lib().exl3_rope(r._ref, _ints(positions, "positions", T, q.device), T, D, _dtype_id(q.dtype, "q"),
                            ctypes.byref(qr), ctypes.byref(qo), kr, ko, _raw_stream(q.device.index)))
    return q_out if k is None else (q_out, k_out)


def _cache_rows(cache: KvCache, t: torch.Tensor, name: str) -> _Rows:
    if t.dtype != cache.dtype or t.device != cache.device or t.shape[-1] != cache.head_dim:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, the cache holds {cache.dtype} heads of "
                         f"{cache.head_dim} on {cache.device}")
    return _rows(t, name)


def cache_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Writes k and v [tokens, heads, head_dim] to the cache's slots (int32 [tokens]; -1: skipped)."""
    if _current_device() != cache.device.index:
        with torch.cuda.device(cache.device):
            return cache_write(cache, k, v, slots)
    kr, vr = _cache_rows(cache, k, "k"), _cache_rows(cache, v, "v")
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"k has {T} tokens, v {v.shape[0]}")
    _check(_lib().exl3_cache_write(cache._ref, ctypes.byref(kr), ctypes.byref(vr),
                                   _ints(slots, "slots", T, cache.device), T, _raw_stream(cache.device.index)))


def rope_cache_write(cache: KvCache, r: Rope, positions: torch.Tensor, slots: torch.Tensor, q: torch.Tensor,
                     k: torch.Tensor, v: torch.Tensor, q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None, norm: Optional[HeadNorm] = None) -> torch.Tensor:
    """rope(q, k) and cache_write(rotated k, v) in one launch, with the same bits; returns the rotated q.  The rotated
    k also goes to k_out when that is given.  norm: q and k are normed per head first, in the same pass."""
    if _current_device() != cache.device.index:
        with torch.cuda.device(cache.device):
            return rope_cache_write(cache, r, positions, slots, q, k, v, q_out, k_out, norm)
    T = q.shape[0]
    qr, kr, vr = _cache_rows(cache, q, "q"), _cache_rows(cache, k, "k"), _cache_rows(cache, v, "v")
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q has {T} tokens, k {k.shape[0]}, v {v.shape[0]}")
    _same_device(r, q)
    q_out, qo = _out(q_out, q, "q_out")
    ko = ctypes.byref(_out(k_out, k, "k_out")[1]) if k_out is not None else None
    if norm is not None or r.axes is not None:
        at, stride = _positions(r, positions, T, q.device)
        _check(_lib().exl3_norm_rope_cache_write(cache._ref, r._axes_ref, _norm(norm, q), at, stride,
                                                 _ints(slots, "slots", T, q.device), T, ctypes.byref(qr), ctypes.byref(qo),
                                                 ctypes.byref(kr), ko, ctypes.byref(vr), _raw_stream(cache.device.index)))
        return q_out
    _check(_lib().exl3_rope_cache_write(cache._ref, r._ref, _ints(positions, "positions", T, q.device),
                                        _ints(slots, "slots", T, q.device), T, ctypes.byref(qr), ctypes.byref(qo),
                                        ctypes.byref(kr), ko, ctypes.byref(vr), _raw_stream(cache.device.index)))
    return q_out


def cache_read(cache: KvCache, slots: torch.Tensor, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values of the slots (int32 [n]) as [n, heads, head_dim] of the cache's dtype; -1 reads as zeros."""
    if _current_device() != cache.device.index:
        with torch.cuda.device(cache.device):
            return cache_read(cache, slots, k_out, v_out)
    n = slots.shape[0]
    shape = (n, cache.heads, cache.head_dim)
    if k_out is None:
        k_out = slots.new_empty(shape, dtype=cache.dtype)
    if v_out is None:
        v_out = torch.empty_like(k_out, memory_format=torch.contiguous_format)
    kr, vr = _cache_rows(cache, k_out, "k_out"), _cache_rows(cache, v_out, "v_out")
    if k_out.shape[0] != n or v_out.shape[0] != n:
        raise ValueError(f"{n} slots, k_out has {k_out.shape[0]} tokens, v_out {v_out.shape[0]}")
    _check(_lib().exl3_cache_read(cache._ref, _ints(slots, "slots", n, cache.device), n, ctypes.byref(kr),
                                  ctypes.byref(vr), _raw_stream(cache.device.index)))
    return k_out, v_out


def attention_workspace_bytes(batch: int, tokens: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """The workspace of an attention call of these sizes, e.g. for reserve_workspace before a capture."""
    L = _lib()
    n = L.exl3_attention_workspace_bytes(batch, tokens, q_heads, kv_heads, head_dim)
    if n == 0 and L.exl3_last_error():
        _check(1)
    return n


def paged_attention(cache: KvCache, q: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor,
                    page_table: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                    out: Optional[torch.Tensor] = None, sinks: int = 0) -> torch.Tensor:
    """Attention of new tokens over the cache, which already holds their own keys and values.

    q [tokens, q_heads, head_dim]: sequence s has rows cu_q[s]..cu_q[s+1]-1 (int32 [batch+1]) and kv_len[s] keys
    (int32 [batch]); its last row is at position kv_len[s]-1.  A row sees the keys up to its own position (window > 0:
    the last `window` of them, and those of the sequence's first `sinks` tokens).  page_table int32 [batch, width]: the
    page of keys j*page_size...; pages that are not the cache's (-1) are holes.  scale defaults to head_dim^-0.5.  Rows that see no key are zero.
    out may be q (in place), and else overlaps neither it nor the cache."""
    if _current_device() != cache.device.index:
        with torch.cuda.device(cache.device):
            return paged_attention(cache, q, cu_q, kv_len, page_table, scale, window, out, sinks)
    T, H, D = q.shape
    B = kv_len.shape[0]
    dev = cache.device
    qr = _cache_rows(cache, q, "q")
    _page_table(page_table, B, dev)
    out, o = _out(out, q, "out")
    L = _lib()
    need = L.exl3_attention_workspace_bytes(B, T, H, cache.heads, D)
    stream = _raw_stream(dev.index)
    ws, wsn = _scratch(need, dev, stream)
    if sinks and _sinks(sinks, window):
        _check(L.exl3_paged_attention_sinks(cache._ref, ctypes.byref(qr), ctypes.byref(o), _ints(cu_q, "cu_q", B + 1, dev),
                                            _ints(kv_len, "kv_len", B, dev), page_table.data_ptr(), page_table.stride(0),
                                            page_table.shape[1], B, T, D ** -0.5 if scale is None else scale,
                                            _window(window), sinks, ws, wsn, stream))
        return out
    _check(L.exl3_paged_attention(cache._ref, ctypes.byref(qr), ctypes.byref(o), _ints(cu_q, "cu_q", B + 1, dev),
                                  _ints(kv_len, "kv_len", B, dev), page_table.data_ptr(), page_table.stride(0),
                                  page_table.shape[1], B, T, D ** -0.5 if scale is None else scale, _window(window), ws, wsn,
                                  stream))
    return out


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True,
                     window: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     sinks: int = 0) -> torch.Tensor:
    """Attention within packed sequences: q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim], sequence
    s the rows cu_seqlens[s]..cu_seqlens[s+1]-1 (int32 [batch+1]).  causal: a row sees the rows of its sequence up to
    itself (window > 0: the last `window` of them, and the sequence's first `sinks` rows), else all.  scale defaults to
    head_dim^-0.5.  out may be q (in place), and else overlaps none of q, k and v."""
    T, H, D = q.shape
    B = cu_seqlens.shape[0] - 1
    qr, kr, vr = _rows(q, "q"), _rows(k, "k", q), _rows(v, "v", q)
    if _current_device() != q.device.index:
        with torch.cuda.device(q.device):
            return prompt_attention(q, k, v, cu_seqlens, causal, window, scale, out, sinks)
    out, o = _out(out, q, "out")
    L = _lib()
    need = L.exl3_attention_workspace_bytes(B, T, H, k.shape[1], D)
    stream = _raw_stream(q.device.index)
    ws, wsn = _scratch(need, q.device, stream)
    if sinks and _sinks(sinks, window) and causal:
        _check(L.exl3_prompt_attention_sinks(ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr), ctypes.byref(o),
                                             _ints(cu_seqlens, "cu_seqlens", B + 1, q.device), B, T, D,
                                             _dtype_id(q.dtype, "q"), _window(window), sinks,
                                             D ** -0.5 if scale is None else scale, ws, wsn, stream))
        return out
    _check(L.exl3_prompt_attention(ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr), ctypes.byref(o),
                                   _ints(cu_seqlens, "cu_seqlens", B + 1, q.device), B, T, D, _dtype_id(q.dtype, "q"),
                                   int(causal), _window(window), D ** -0.5 if scale is None else scale, ws, wsn, stream))
    return out


def prefix_attention_workspace_bytes(batch: int, tokens: int, groups: int, q_heads: int, kv_heads: int,
                                     head_dim: int) -> int:
    """The workspace of a prefix_attention call of these sizes, e.g. for reserve_workspace before a capture."""
    L = _lib()
    n = L.exl3_prefix_attention_workspace_bytes(batch, tokens, groups, q_heads, kv_heads, head_dim)
    if n == 0 and L.exl3_last_error():
        _check(1)
    return n


def prefix_attention(cache: KvCache, q: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor,
                     page_table: torch.Tensor, group_cu: torch.Tensor, prefix_len: torch.Tensor,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention of sequences that share prefixes, whose keys and values are read once for all that share them.

    Group g is the sequences group_cu[g]..group_cu[g+1]-1 (int32 [groups+1]); their rows of the page table have the same
    pages for their first prefix_len[g] keys (int32 [groups]; rows of sequences without new tokens may hold anything).
    Sequences of no group share nothing.  The rest is paged_attention's, and so is the result but for the order of
    sums.  Whether sharing is worth its passes is decided by the sizes, a page table counting as full to its width: one
    much wider than the sequences makes short calls slower (18 us instead of 11).  The workspace (up to 1 GiB more than
    paged_attention's) is kept for the stream."""
    if _current_device() != cache.device.index:
        with torch.cuda.device(cache.device):
            return prefix_attention(cache, q, cu_q, kv_len, page_table, group_cu, prefix_len, scale, out)
    T, H, D = q.shape
    B, G = kv_len.shape[0], prefix_len.shape[0]
    dev = cache.device
    qr = _cache_rows(cache, q, "q")
    _page_table(page_table, B, dev)
    out, o = _out(out, q, "out")
    L = _lib()
    need = L.exl3_prefix_attention_workspace_bytes(B, T, G, H, cache.heads, D)
    stream = _raw_stream(dev.index)
    ws, wsn = _scratch(need, dev, stream)
    _check(L.exl3_prefix_attention(cache._ref, ctypes.byref(qr), ctypes.byref(o), _ints(cu_q, "cu_q", B + 1, dev),
                                   _ints(kv_len, "kv_len", B, dev), page_table.data_ptr(), page_table.stride(0),
                                   page_table.shape[1], B, T, _ints(group_cu, "group_cu", G + 1, dev),
                                   _ints(prefix_len, "prefix_len", G, dev), G, D ** -0.5 if scale is None else scale,
                                   ws, wsn, stream))
    return out


class CacheStep(NamedTuple):
    """A step's rows of requests over the cache, int32 on the GPU (cache_extend)."""

    cu_q: torch.Tensor       # [batch+1] request b's rows are cu_q[b]..cu_q[b+1]-1
    kv_len: torch.Tensor     # [batch] tokens in the cache with the step's own
    positions: torch.Tensor  # [tokens] of each row (0 where no request has it)
    slots: torch.Tensor      # [tokens] in the cache (-1 where there is none)
    counts: torch.Tensor     # [2] the rows that were wanted, and the pages that were needed


def _page_table(page_table: torch.Tensor, batch: int, device) -> None:
    if (page_table.dtype != torch.int32 or page_table.device != device or page_table.dim() != 2 or
            page_table.shape[0] != batch or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError(f"page_table must be int32 [{batch}, width] with dense rows on {device}, got {page_table.dtype} "
                         f"{tuple(page_table.shape)}")


def cache_extend(cache: KvCache, q_len: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor,
                 free_pages: torch.Tensor, tokens: int, taken: Optional[torch.Tensor] = None,
                 out: Optional[CacheStep] = None) -> CacheStep:
    """What a step needs of its requests' lengths, in one launch that reads nothing back: request b has kv_len[b] tokens
    in the cache and wants q_len[b] more (int32 [batch]), of `tokens` rows that the requests get in order.

    page_table (int32 [batch, width]) gets the pages that the new tokens need, from free_pages (int32 [n]) in the
    requests' order, from place taken[0] on (int32 [1]; None: from the first); -1 where none is left.  Returns the rows'
    offsets, the new lengths, and each row's position and slot, in new tensors or those of `out`, which overlap no input;
    counts[1] is what the step took of free_pages, or more if they were too few.  Rows that no request has (a step of
    fixed size) have slot -1, and so do those without a page.  A request that wants more rows than are left gets those:
    counts[0] is then more than `tokens`."""
    dev = cache.device
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return cache_extend(cache, q_len, kv_len, page_table, free_pages, tokens, taken, out)
    B = kv_len.shape[0]
    _page_table(page_table, B, dev)
    if not 0 <= tokens <= 1 << 20:
        raise ValueError(f"tokens={tokens}, must be 0 to {1 << 20}")
    at = [_ints(q_len, "q_len", B, dev), _ints(kv_len, "kv_len", B, dev)]
    free_at = _ints(free_pages, "free_pages", free_pages.shape[0], dev)
    taken_at = None if taken is None else _ints(taken, "taken", 1, dev)
    sizes = (B + 1, B, tokens, tokens, 2)
    if out is None:
        new = kv_len.new_empty(2 * B + 3 + 2 * tokens)  # all of them are views of it
        out, a = CacheStep(*new.split(sizes)), new.data_ptr()
        made = (a, a + 4 * (B + 1), a + 4 * (2 * B + 1), a + 4 * (2 * B + 1 + tokens), a + 4 * (2 * B + 1 + 2 * tokens))
    else:
        made = [_ints(t, name, n, dev) for t, name, n in zip(out, CacheStep._fields, sizes)]
    _check(_lib().exl3_cache_extend(cache.pages, cache.page_size, *at, B, page_table.data_ptr(), page_table.stride(0),
                                    page_table.shape[1], free_at, free_pages.shape[0], taken_at, tokens, *made,
                                    _raw_stream(dev.index)))
    return out
