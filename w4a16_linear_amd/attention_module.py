"""A self-attention layer of a served transformer on libopq's kernels, end to end:
OPQ-quantized QKV projection, rotary positions on queries and keys in one call, keys
and values quantized into the paged cache, attention of the new tokens (one per
sequence, a chain, or a tree of drafted ones) over it, OPQ-quantized output projection.

    layer = OPQAttention(3840, heads=30, kv_heads=30).to(torch.bfloat16).cuda()
    replace_with_opq(layer)                      # quantize both projections
    cache = layer.new_cache(pages=512, page=64, fmt="opq4")
    y = layer(x, cache, page_table, lens)        # x [batch, draft, hidden]
    layer.accept(cache, page_table, lens, kept)  # of a verified tree

Every step but the projections' reshapes runs in libopq; like OPQLinear, a layer whose
tensors are not on the GPU raises.  No gradient passes through the cache: where one would
be lost (x or qkv's weights require it and gradients are on) a forward raises.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import torch
from torch import nn

from . import attention as A


def token_slots(page_table: torch.Tensor, positions: torch.Tensor, page: int,
                pages: Optional[int] = None) -> torch.Tensor:
    """Cache slots (int32, the shape of `positions` [batch, n]) of positions in each
    sequence; -1 (no slot) past the page table, for negative positions, and where the page
    id is none of the cache's `pages` (not given: of as many as a cache can have, fewer than
    2^31 tokens: a larger id must not wrap around to another page's slots)."""
    if page_table.shape[1] == 0 or pages == 0:   # nothing to look up, no index that is inside
        return torch.full_like(positions, -1, dtype=torch.int32)
    index = torch.div(positions, page, rounding_mode="floor")
    at = index.clamp(0, page_table.shape[1] - 1)
    ids = torch.gather(page_table, 1, at.long())
    last = ((2 ** 31 - 1) // page if pages is None else pages) - 1
    inside = (index == at) & (ids == ids.clamp(0, last))
    return torch.where(inside, ids * page + positions % page, -1).to(torch.int32)


def _int32(name: str, t: torch.Tensor, shape, device: torch.device, dense: bool = True) -> None:
    if t.dtype != torch.int32 or t.shape != shape or t.device != device or (dense and not t.is_contiguous()):
        raise ValueError(f"{name} must be{' contiguous' if dense else ''} int32 {shape} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


class OPQAttention(nn.Module):
    """`qkv` [hidden -> (heads + 2 kv_heads) dim] and `o` [heads dim -> hidden] start as
    nn.Linear (replace_with_opq makes them OPQLinear); the rotary table, `rope`, covers
    max_positions.  dim is hidden / heads unless given; 64, 128 or 256."""

    def __init__(self, hidden: int, heads: int, kv_heads: Optional[int] = None,
                 dim: Optional[int] = None, max_positions: int = 32768, rot: Optional[int] = None,
                 base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 original_len: float = 0.0, layout: str = "half"):
        super().__init__()
        self.hidden, self.heads, self.kv_heads = hidden, heads, kv_heads or heads
        self.dim = dim or hidden // heads
        if self.heads % self.kv_heads:
            raise ValueError(f"heads={heads} must be a multiple of kv_heads={kv_heads}")
        if self.dim not in (64, 128, 256):
            raise ValueError(f"dim must be 64, 128 or 256, got {self.dim}")
        self.layout, self.max_positions = layout, max_positions
        self.frequencies = A.rotary_frequencies(rot or self.dim, base, scaling, factor, original_len)
        self.qkv = nn.Linear(hidden, (self.heads + 2 * self.kv_heads) * self.dim, bias=False)
        self.o = nn.Linear(self.heads * self.dim, hidden, bias=False)
        self._ropes: Dict[torch.device, torch.Tensor] = {}   # float32 whatever the layer's type

    def rope(self, device: torch.device) -> torch.Tensor:
        """The rotary table on `device`, made at the first call there and kept.  That call
        waits for it, so that every stream and thread may use what is kept without asking
        who made it; it cannot be part of a graph's capture."""
        table = self._ropes.get(device)
        if table is None:   # a name, or the first call
            device = torch.device(device)
            if device.type == "cuda" and device.index is None:
                device = torch.device("cuda", torch.cuda.current_device())
            table = self._ropes.get(device)
        if table is None:
            if device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the layer's rotary table is not made yet: call rope(device), or run the "
                                   "layer once, before capturing it in a graph")
            table = A.rotary_table(self.frequencies, self.max_positions, device)
            torch.cuda.current_stream(device).synchronize()
            self._ropes[device] = table
        return table

    def new_cache(self, pages: int, page: int = 64, fmt: str = "opq4", alpha: float = 0.73,
                  device="cuda") -> A.PagedCache:
        return A.new_cache(pages, self.kv_heads, page, self.dim, fmt, alpha, device)

    def _check(self, x, cache, page_table, lens, mask, depths, counts, max_len) -> None:
        """All that the calls of a forward would refuse, before the first of them writes (a
        few microseconds: a step of one token is not much more on the host)."""
        if x.dim() != 3 or x.shape[2] != self.hidden or x.dtype != torch.bfloat16:
            raise ValueError(f"x must be bfloat16 [batch, draft, {self.hidden}], got {x.dtype} {tuple(x.shape)}")
        # qkv's own weights; those of modules inside it are met at rotary, before anything is written
        if torch.is_grad_enabled() and (x.requires_grad or any(
                w is not None and w.requires_grad for w in self.qkv._parameters.values())):
            raise RuntimeError("this layer serves and passes no gradients back: call it under torch.no_grad(), "
                               "or with x and the weights of qkv not requiring them")
        batch, draft, _ = x.shape
        _, heads, page = cache.k_scale.shape
        if heads != self.kv_heads or cache.dim != self.dim:
            raise ValueError(f"the cache has {heads} heads of {cache.dim}, the layer {self.kv_heads} of {self.dim}")
        device, columns = x.device, page_table.shape[-1]
        _int32("page_table", page_table, (batch, columns), device)
        _int32("lens", lens, (batch,), device)
        if mask is not None:
            words = (draft, (draft + 31) // 32)
            _int32("mask", mask, words if mask.dim() == 2 else (batch,) + words, device)
        if depths is not None:   # only enters a sum here; the others' memory goes to the kernels
            _int32("depths", depths, (batch, draft), device, dense=False)
        if counts is not None:
            _int32("counts", counts, (batch,), device)
        if max_len is not None and not 0 <= max_len <= columns * page:
            raise ValueError(f"max_len must be 0 to {columns * page}, what the page table holds, got {max_len}")

    def forward(self, x: torch.Tensor, cache: A.PagedCache, page_table: torch.Tensor,
                lens: torch.Tensor, mask: Optional[torch.Tensor] = None,
                depths: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                max_len: Optional[int] = None) -> torch.Tensor:
        """x [batch, draft, hidden] (bfloat16): the tokens after each sequence's lens[b]
        cached ones, written to the cache here.  mask: tree words as tree_attention
        takes them, and with it depths (int32 [batch, draft]): each token's distance from the
        last cached one, less one, which gives its position; without a mask a chain."""
        if mask is not None and depths is None:
            raise ValueError("a mask needs depths: a tree's tokens are not at the positions of their places")
        self._check(x, cache, page_table, lens, mask, depths, counts, max_len)
        batch, draft, _ = x.shape
        pages, _, page = cache.k_scale.shape
        rope = self.rope(x.device)
        places = lens[:, None]                               # where tokens are stored
        if draft != 1 or counts is not None:
            steps = torch.arange(draft, dtype=torch.int32, device=x.device)
            places = places + steps
        positions = places if depths is None else lens[:, None] + depths
        if counts is not None:
            places = torch.where(steps < counts[:, None], places, -1)
        slots = token_slots(page_table, places, page, pages)
        h, k = self.heads, self.kv_heads
        fused = self.qkv(x).view(batch * draft, h + 2 * k, self.dim)
        qk = fused[:, :h + k]
        A.rotary(qk, positions.reshape(-1).contiguous(), rope, self.layout, out=qk)
        A.cache_write(cache, fused[:, h:h + k], fused[:, h + k:], slots.reshape(-1))
        q = fused.view(batch, draft, h + 2 * k, self.dim)[:, :, :h]
        y = A.tree_attention(q, cache, page_table, lens, mask=mask, counts=counts, max_len=max_len)
        return self.o(y.view(batch, draft, h * self.dim))

    @staticmethod
    def accept(cache: A.PagedCache, page_table: torch.Tensor, lens: torch.Tensor,
               kept: torch.Tensor) -> None:
        """Keep a path of a verified tree: kept int32 [batch, n] holds the accepted drafted
        tokens' indexes in order (-1 past a path's end); they move up to positions
        lens[b], lens[b] + 1, ...  The caller adds the path's length to lens."""
        n = torch.arange(kept.shape[1], dtype=torch.int32, device=kept.device)
        src = torch.where(kept >= 0, lens[:, None] + kept, -1)
        dst = torch.where(kept >= 0, lens[:, None] + n, -1)
        A.cache_move(cache, token_slots(page_table, src, cache.page, cache.pages).contiguous(),
                     token_slots(page_table, dst, cache.page, cache.pages).contiguous())


__all__: Sequence[str] = ["OPQAttention", "token_slots"]
