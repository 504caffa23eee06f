"""Python binding of libopq's attention side (include/opq_attention.h): rotary
positions, a paged key/value cache quantized as it is written, and attention of
drafted tokens (one, or a tree of them, per sequence) over that cache.

As in ``opq``, tensors are checked, outputs are allocated with torch on the
caller's device, and raw pointers go to the library with the current torch stream;
every step runs in its HIP kernels.  For the calls of a decode step, where Python
would take longer than the GPU, this is done in C++ (csrc/attention_torch.cpp, built
as _attention.so).  Workspaces come from torch's allocator per call, so calls on
different streams do not share one.

Only apply_rotary is followed by autograd.  Every other call refuses (RuntimeError) a
tensor that requires grad unless gradients are off (torch.no_grad()), rather than
return a result cut off from it.

    table = rotary_table(rotary_frequencies(128, 1e6), 32768, "cuda")
    cache = new_cache(pages=1024, heads=8, page=64, dim=128, fmt="opq4", device="cuda")
    qk = rotary(qkv.view(tokens, 48, 128)[:, :40], positions, table)
    cache_write(cache, qk[:, 32:], v, slots)
    out = tree_attention(qk[:, :32].view(batch, draft, 32, 128), cache, page_table, lens, mask)
"""
from __future__ import annotations

import ctypes
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
    "opq_cache_move": (_I, [_P, _L, _L, _P, _P, _P]),
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
_ext = None


def load() -> ctypes.CDLL:
    """libopq.so with the attention side's signatures set, and the extension that takes
    tensors to it; raises if either is missing."""
    global _ready, _ext
    if _ready is None:
        lib = opq.load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        try:
            from . import _attention
        except ImportError as e:
            raise RuntimeError("_attention.so not built: run `python -m w4a16_linear_amd.build`") from e
        _attention.set_error(opq.OpqError)
        _ext = _attention
        _ready = lib
    return _ready


def _calls():
    if _ext is None:
        load()
    return _ext


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
    with torch.cuda.device(f.device):
        stream = torch.cuda.current_stream(f.device).cuda_stream
        _check("opq_rotary_table",
               load().opq_rotary_table(f.data_ptr(), f.numel(), length,
                                       1.0 if amplitude is None else amplitude, table.data_ptr(),
                                       stream))
    return table


def _rotary(x, positions, table, layout, sections, out, backward):
    code = LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {list(LAYOUTS)}, got {layout!r}")
    return (_ext or _calls()).rotary(x, positions, table, code, sections, out, backward)


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
    """The turn one way; its gradient is the turn the other way, an operation of its own,
    so gradients of gradients are followed too."""

    @staticmethod
    def forward(ctx, x, positions, table, layout, sections, backward):
        ctx.save_for_backward(positions, table)
        ctx.how = (layout, sections, not backward)
        return _rotary(x, positions, table, layout, sections, None, int(backward))

    @staticmethod
    def backward(ctx, grad):
        positions, table = ctx.saved_tensors
        if grad.shape[-1] > 1 and grad.stride(-1) != 1:
            grad = grad.contiguous()
        return _Rotary.apply(grad, positions, table, *ctx.how), None, None, None, None, None


def apply_rotary(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, layout: str = "half",
                 sections: Optional[Sequence[int]] = None) -> torch.Tensor:
    """rotary() that autograd differentiates with respect to x, as often as asked (not with
    respect to the table)."""
    if table.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("table requires grad, which apply_rotary does not follow: detach it")
    return _Rotary.apply(x, positions, table, layout, None if sections is None else tuple(sections), False)


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


def cache_write(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k, v [tokens, heads, dim] (float32 or bfloat16; token and head
    strides free) into the rows of `slots` (int32 [tokens]; -1 skips a token)."""
    (_ext or _calls()).cache_write(cache, k, v, slots)


def cache_read(cache: PagedCache, slots: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, heads, dim] of the rows of `slots` (int32 [tokens]; -1
    gives zeros), as bfloat16 or float32."""
    dtype = _DTYPES.get(out_dtype)
    if dtype is None:
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    k, v = (None, None) if out is None else out
    return (_ext or _calls()).cache_read(cache, slots, dtype, k, v)


def cache_move(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Move rows as they are stored from slots src to slots dst (int32 [batch,
    count], count up to 128; -1 moves nothing): the accepted tokens of a verified tree
    to the slots right after the cached ones.  A sequence's rows are all read before
    any is written; sequences of one call must not share slots."""
    (_ext or _calls()).cache_move(cache, src, dst)


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
    return (_ext or _calls()).attention(q, cache, page_table, lens, mask, counts, scale, max_len, out,
                                        return_lse, workspace)


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
