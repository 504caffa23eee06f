"""Python binding of libopq's attention side (include/opq_attention.h): rotary
positions, a paged key/value cache quantized as it is written, and attention of
drafted tokens (one, or a tree of them, per sequence) over that cache.

As in ``opq``, this module checks tensors, allocates outputs with torch on the
caller's device and passes raw pointers plus the current torch stream; every step
runs in the library's HIP kernels.  Workspaces come from torch's allocator per
call, so calls on different streams do not share one.

    table = rotary_table(rotary_frequencies(128, 1e6), 32768, "cuda")
    cache = new_cache(pages=1024, heads=8, page=64, dim=128, fmt="opq4", device="cuda")
    qk = rotary(qkv.view(tokens, 48, 128)[:, :40], positions, table)
    cache_write(cache, qk[:, 32:], v, slots)
    out = tree_attention(qk[:, :32].view(batch, draft, 32, 128), cache, page_table, lens, mask)
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple, Optional, Sequence, Tuple

import numpy as np
import torch

from . import opq
from .opq import OPQ_BF16, OPQ_F32, _check

_P, _I, _L, _F, _D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                      ctypes.c_double)

# signatures in header order
_SIGNATURES = {
    "opq_rotary_frequencies": (_I, [_L, _D, _I, _D, _D, _D, _D, _P, _P]),
    "opq_rotary_table": (_I, [_P, _L, _L, _D, _P, _P]),
    "opq_rotary": (_I, [_P, _I, _L, _L, _L, _L, _L, _P, _L, _P, _P, _L, _L, _I, _I, _P, _L, _L, _P]),
    "opq_cache_write": (_I, [_P, _P, _L, _L, _P, _L, _L, _I, _L, _P, _P]),
    "opq_cache_read": (_I, [_P, _L, _P, _P, _P, _I, _P]),
    "opq_cache_attention_workspace_bytes": (ctypes.c_size_t, [_L, _L, _L, _L, _L, _L]),
    "opq_cache_attention": (_I, [_P, _P, _L, _L, _L, _L, _L, _L, _P, _L, _P, _P, _L, _P, _L, _F,
                                 _P, _P, _P, ctypes.c_size_t, _P]),
}

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
FORMATS = {"bf16": 0, "fp8": 1, "opq4": 2}
_CODE_TYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "opq4": torch.int32}
_DTYPES = {torch.float32: OPQ_F32, torch.bfloat16: OPQ_BF16}


class _CCache(ctypes.Structure):
    _fields_ = [("k", _P), ("k_sign", _P), ("k_scale", _P), ("v", _P), ("v_sign", _P),
                ("v_scale", _P), ("pages", _L), ("heads", _L), ("page", _L), ("dim", _L),
                ("format", _I), ("alpha", _F)]


_ready: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """libopq.so with the attention side's signatures set."""
    global _ready
    if _ready is None:
        lib = opq.load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _ready = lib
    return _ready


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, shape: Tuple[int, ...]) -> int:
    """Checks a dense device tensor of a known shape; returns its address."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _need_rows(name: str, t: torch.Tensor, ndim: int, like: Optional[torch.device] = None) -> None:
    """Checks a device tensor whose last dimension is dense; other strides are free."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != ndim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be {ndim}-d with a dense last dimension")
    if like is not None and t.device != like:
        raise ValueError(f"{name} must be on {like}, got {t.device}")


def _same_device(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


class _on:
    """The library launches on the current device: make it the tensors' one."""

    __slots__ = ("dev", "old")

    def __init__(self, dev: torch.device):
        self.dev = dev.index

    def __enter__(self) -> int:
        self.old = torch.cuda.current_device()
        if self.old != self.dev:
            torch.cuda.set_device(self.dev)
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc) -> None:
        if self.old != self.dev:
            torch.cuda.set_device(self.old)


# ------------------------------------------------------------------ rotary

class RotaryFrequencies(NamedTuple):
    freq: np.ndarray   # float64 [rot/2], radians per position
    amplitude: float   # factor of cos and sin


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None,
                       factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0,
                       beta_slow: float = 1.0) -> RotaryFrequencies:
    """Frequencies of `rot` turned dimensions (host).  `scaling` stretches them
    for contexts `factor` times as long: "linear" (positions interpolated),
    "ntk" (a larger base) or "yarn" (slow pairs interpolated, fast ones kept,
    counted in turns over `original_len` positions; with its amplitude)."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {list(SCALINGS)}, got {scaling!r}")
    f = np.zeros(max(1, rot // 2), np.float64)
    amp = ctypes.c_double(1.0)
    _check("opq_rotary_frequencies",
           load().opq_rotary_frequencies(rot, base, SCALINGS[scaling], factor, original_len,
                                         beta_fast, beta_slow, f.ctypes.data, ctypes.byref(amp)))
    return RotaryFrequencies(f, amp.value)


def rotary_table(frequencies, length: int, device, amplitude: Optional[float] = None) -> torch.Tensor:
    """float32 [length, pairs, 2]: amplitude * (cos, sin) of every position.
    `frequencies` is what rotary_frequencies gives or a float64 array [pairs]
    (for several position axes: theirs, one after the other)."""
    if isinstance(frequencies, RotaryFrequencies):
        amplitude = frequencies.amplitude if amplitude is None else amplitude
        frequencies = frequencies.freq
    f = torch.as_tensor(np.ascontiguousarray(frequencies, np.float64)).to(device)
    if f.dim() != 1 or not f.is_cuda:
        raise ValueError("frequencies must be one row, and device a CUDA (HIP) device")
    table = torch.empty((length, f.numel(), 2), dtype=torch.float32, device=f.device)
    with _on(f.device) as stream:
        _check("opq_rotary_table",
               load().opq_rotary_table(f.data_ptr(), f.numel(), length,
                                       1.0 if amplitude is None else amplitude, table.data_ptr(),
                                       stream))
    return table


@lru_cache(maxsize=64)
def _sections(sections: Tuple[int, ...]):
    return (ctypes.c_int32 * len(sections))(*sections)


def _rotary(x, positions, table, layout, sections, out, backward):
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {list(LAYOUTS)}, got {layout!r}")
    _need_rows("x", x, 3)
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    tokens, heads, dim = x.shape
    if table.dim() != 3:
        raise ValueError("table must be [length, pairs, 2]")
    pairs = table.shape[1]
    pt = _need("table", table, torch.float32, (table.shape[0], pairs, 2))
    sections = (pairs,) if sections is None else tuple(sections)
    axes = len(sections)
    if positions.dim() == 1 and axes == 1:
        positions = positions.unsqueeze(1)
    pp = _need("positions", positions, torch.int32, (tokens, axes))
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=x.dtype, device=x.device)
    else:
        _need_rows("out", out, 3)
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError(f"out must be {x.dtype} of shape {tuple(x.shape)}")
    _same_device(x.device, positions=positions, table=table, out=out)
    xs, os = x.stride(), out.stride()
    with _on(x.device) as stream:
        st = load().opq_rotary(x.data_ptr(), _DTYPES[x.dtype], tokens, heads, dim, xs[0], xs[1], pp,
                               axes, _sections(sections), pt, table.shape[0], 2 * pairs,
                               LAYOUTS[layout], backward, out.data_ptr(), os[0], os[1], stream)
    _check("opq_rotary", st)
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, layout: str = "half",
           sections: Optional[Sequence[int]] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [tokens, heads, dim] (float32 or bfloat16; token and head strides free)
    with the first 2 * table.shape[1] dimensions of every head turned to the
    tokens' positions: int32 [tokens], or [tokens, axes] with `sections` pairs
    per axis.  `out` may be x itself."""
    return _rotary(x, positions, table, layout, sections, out, 0)


def rotary_backward(grad: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
                    layout: str = "half", sections: Optional[Sequence[int]] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of rotary's x from the gradient of its result."""
    return _rotary(grad, positions, table, layout, sections, out, 1)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, table, layout, sections):
        ctx.save_for_backward(positions, table)
        ctx.how = (layout, sections)
        return rotary(x, positions, table, layout, sections)

    @staticmethod
    def backward(ctx, grad):
        positions, table = ctx.saved_tensors
        if grad.shape[-1] > 1 and grad.stride(-1) != 1:
            grad = grad.contiguous()
        return rotary_backward(grad, positions, table, *ctx.how), None, None, None, None


def apply_rotary(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, layout: str = "half",
                 sections: Optional[Sequence[int]] = None) -> torch.Tensor:
    """rotary() that autograd differentiates with respect to x."""
    return _Rotary.apply(x, positions, table, layout, None if sections is None else tuple(sections))


# ------------------------------------------------------------------- cache

class PagedCache(NamedTuple):
    """A paged key/value cache (include/opq_attention.h: opq_cache).  One row per
    (page, head, offset) and side; slot = page id * page size + offset."""
    fmt: str                          # "bf16", "fp8" or "opq4"
    alpha: float                      # power of "opq4" codes
    k: torch.Tensor                   # [pages, heads, page, dim] bfloat16 / float8_e4m3fn,
                                      # [pages, heads, page, dim/8] int32 for "opq4"
    k_sign: Optional[torch.Tensor]    # "opq4": int32 [pages, heads, page, dim/32]
    k_scale: torch.Tensor             # float32 [pages, heads, page]
    v: torch.Tensor
    v_sign: Optional[torch.Tensor]
    v_scale: torch.Tensor

    @property
    def pages(self) -> int:
        return self.k_scale.shape[0]

    @property
    def heads(self) -> int:
        return self.k_scale.shape[1]

    @property
    def page(self) -> int:
        return self.k_scale.shape[2]

    @property
    def dim(self) -> int:
        return self.k.shape[3] * (8 if self.fmt == "opq4" else 1)

    @property
    def device(self) -> torch.device:
        return self.k.device


def new_cache(pages: int, heads: int, page: int, dim: int, fmt: str = "fp8", alpha: float = 0.73,
              device="cuda") -> PagedCache:
    """An empty cache (zeros: every row reads as 0)."""
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {list(FORMATS)}, got {fmt!r}")
    if dim not in (64, 128, 256):
        raise ValueError(f"dim must be 64, 128 or 256, got {dim}")
    if page < 16 or page & (page - 1):
        raise ValueError(f"page must be a power of two, 16 or more, got {page}")

    def side():
        words = dim // 8 if fmt == "opq4" else dim
        codes = torch.zeros((pages, heads, page, words), device=device,
                            dtype=torch.uint8 if fmt == "fp8" else _CODE_TYPES[fmt])
        sign = torch.zeros((pages, heads, page, dim // 32), dtype=torch.int32,
                           device=device) if fmt == "opq4" else None
        return (codes.view(torch.float8_e4m3fn) if fmt == "fp8" else codes, sign,
                torch.zeros((pages, heads, page), dtype=torch.float32, device=device))

    return PagedCache(fmt, alpha, *side(), *side())


def _c_cache(cache: PagedCache) -> _CCache:
    fmt = cache.fmt
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {list(FORMATS)}, got {fmt!r}")
    if cache.k.dim() != 4:
        raise ValueError("cache codes must be [pages, heads, page, ...]")
    pages, heads, page, words = cache.k.shape
    dt = _CODE_TYPES[fmt]
    shape, rows = (pages, heads, page, words), (pages, heads, page)
    ks = vs = None
    dim = words
    if fmt == "opq4":
        dim = 8 * words
        signs = (pages, heads, page, dim // 32)
        ks = _need("k_sign", cache.k_sign, torch.int32, signs)
        vs = _need("v_sign", cache.v_sign, torch.int32, signs)
        _same_device(cache.k.device, k_sign=cache.k_sign, v_sign=cache.v_sign)
    _same_device(cache.k.device, k_scale=cache.k_scale, v=cache.v, v_scale=cache.v_scale)
    return _CCache(_need("k", cache.k, dt, shape), ks,
                   _need("k_scale", cache.k_scale, torch.float32, rows),
                   _need("v", cache.v, dt, shape), vs,
                   _need("v_scale", cache.v_scale, torch.float32, rows),
                   pages, heads, page, dim, FORMATS[fmt], cache.alpha)


def cache_write(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k, v [tokens, heads, dim] (float32 or bfloat16; token and head
    strides free) into the rows of `slots` (int32 [tokens]; -1 skips a token)."""
    cc = _c_cache(cache)
    _need_rows("k", k, 3, cache.device)
    _need_rows("v", v, 3, cache.device)
    tokens = k.shape[0]
    if k.dtype not in _DTYPES or v.dtype != k.dtype:
        raise ValueError(f"k and v must both be float32 or bfloat16, got {k.dtype} and {v.dtype}")
    if k.shape != v.shape or tuple(k.shape[1:]) != (cc.heads, cc.dim):
        raise ValueError(f"k and v must be [tokens, {cc.heads}, {cc.dim}], got {tuple(k.shape)} "
                         f"and {tuple(v.shape)}")
    sp = _need("slots", slots, torch.int32, (tokens,))
    _same_device(cache.device, slots=slots)
    a, b = k.stride(), v.stride()
    with _on(cache.device) as stream:
        st = load().opq_cache_write(ctypes.byref(cc), k.data_ptr(), a[0], a[1], v.data_ptr(), b[0],
                                    b[1], _DTYPES[k.dtype], tokens, sp, stream)
    _check("opq_cache_write", st)


def cache_read(cache: PagedCache, slots: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, heads, dim] of the rows of `slots` (int32 [tokens]; -1
    gives zeros), as bfloat16 or float32."""
    cc = _c_cache(cache)
    if out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    shape = (slots.shape[0], cc.heads, cc.dim)
    sp = _need("slots", slots, torch.int32, shape[:1])
    if out is None:
        out = (torch.empty(shape, dtype=out_dtype, device=cache.device),
               torch.empty(shape, dtype=out_dtype, device=cache.device))
    kp, vp = _need("out[0]", out[0], out_dtype, shape), _need("out[1]", out[1], out_dtype, shape)
    _same_device(cache.device, slots=slots, k_out=out[0], v_out=out[1])
    with _on(cache.device) as stream:
        st = load().opq_cache_read(ctypes.byref(cc), shape[0], sp, kp, vp, _DTYPES[out_dtype], stream)
    _check("opq_cache_read", st)
    return out[0], out[1]


# --------------------------------------------------------------- attention

def attention_workspace_bytes(batch: int, draft: int, heads: int, kv_heads: int, dim: int,
                              max_len: int) -> int:
    return int(load().opq_cache_attention_workspace_bytes(batch, draft, heads, kv_heads, dim, max_len))


def tree_attention(q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor, lens: torch.Tensor,
                   mask: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, max_len: Optional[int] = None,
                   out: Optional[torch.Tensor] = None, return_lse: bool = False,
                   workspace: Optional[torch.Tensor] = None):
    """Attention of q [batch, draft, heads, dim] (bfloat16) over the cache: each
    sequence's first lens[b] tokens, and its drafted ones as `mask` allows.

    The drafted tokens' keys and values are written already, at positions
    lens[b] .. lens[b] + draft - 1 of the sequence.  page_table: int32 [batch,
    max_pages]; lens: int32 [batch].  mask: int32 [batch, draft, ceil(draft/32)]
    words (or without the batch dimension), bit j of row t set where drafted
    token t sees drafted token j (tree_mask makes them from parents); without a
    mask the draft is a chain.  counts: int32 [batch], drafted tokens that count.
    scale: 1/sqrt(dim) by default.  max_len: an upper bound of lens that the
    caller knows; it sizes the split of the work (default: what the page table
    holds less the draft).  Returns bfloat16 [batch, draft, heads, dim], with
    return_lse also float32 [batch, draft, heads].
    """
    cc = _c_cache(cache)
    dev = cache.device
    _need_rows("q", q, 4, dev)
    if q.dtype != torch.bfloat16:
        raise ValueError(f"q must be bfloat16, got {q.dtype}")
    batch, draft, heads, dim = q.shape
    if dim != cc.dim or heads % cc.heads:
        raise ValueError(f"q has {heads} heads of {dim}, the cache {cc.heads} of {cc.dim}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    max_pages = page_table.shape[1]
    tp = _need("page_table", page_table, torch.int32, (batch, max_pages))
    lp = _need("lens", lens, torch.int32, (batch,))
    mp, mask_batch = None, 0
    if mask is not None:
        words = (draft + 31) // 32
        mask_batch = draft * words if mask.dim() == 3 else 0
        mp = _need("mask", mask, torch.int32,
                   (batch, draft, words) if mask.dim() == 3 else (draft, words))
    cp = None if counts is None else _need("counts", counts, torch.int32, (batch,))
    _same_device(dev, page_table=page_table, lens=lens, mask=mask, counts=counts)
    if max_len is None:
        max_len = max(0, max_pages * cc.page - draft)
    if out is None:
        out = torch.empty((batch, draft, heads, dim), dtype=torch.bfloat16, device=dev)
    else:
        _need("out", out, torch.bfloat16, (batch, draft, heads, dim))
        _same_device(dev, out=out)
    lse = torch.empty((batch, draft, heads), dtype=torch.float32, device=dev) if return_lse else None
    lib = load()
    need = lib.opq_cache_attention_workspace_bytes(batch, draft, heads, cc.heads, dim, max_len)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not workspace.is_cuda or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    s = q.stride()
    with _on(dev) as stream:
        st = lib.opq_cache_attention(
            ctypes.byref(cc), q.data_ptr(), batch, draft, heads, s[0], s[1], s[2], tp, max_pages, lp,
            cp, max_len, mp, mask_batch, dim ** -0.5 if scale is None else scale, out.data_ptr(),
            None if lse is None else lse.data_ptr(),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(), stream)
    _check("opq_cache_attention", st)
    return (out, lse) if return_lse else out


def tree_mask(parents: torch.Tensor) -> torch.Tensor:
    """Mask words int32 [batch, draft, ceil(draft/32)] of trees given by parents
    int32 [batch, draft] on the host (parent index, or -1 under the cached
    tokens; a parent comes before its children): every token sees itself and
    the drafted tokens above it."""
    p = parents.cpu().numpy()
    if p.ndim != 2:
        raise ValueError("parents must be [batch, draft]")
    batch, draft = p.shape
    if ((p >= np.arange(draft)) | (p < -1)).any():
        raise ValueError("a parent must be -1 or come before its child")
    words = np.zeros((batch, draft, (draft + 31) // 32), np.uint32)
    b = np.arange(batch)
    for t in range(draft):
        above = p[:, t]
        words[:, t] = np.where(above[:, None] >= 0, words[b, np.maximum(above, 0)], 0)
        words[:, t, t // 32] |= np.uint32(1 << (t % 32))
    return torch.from_numpy(words.view(np.int32))
