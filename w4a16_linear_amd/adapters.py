"""Python binding of libopq's adapters (include/opq_adapters.h): low-rank adapters of many
requests beside one shared projection, their gradients, and the gradient through a quantized
projection.

As in ``attention``, tensors are checked, outputs are allocated with torch on the caller's
device, and raw pointers go to the library with the current torch stream; workspaces come
from torch's allocator per call, so calls on different streams do not share one.

    stack = Adapters(down, up, scale)             # of one projection, every customer's
    y = opq.linear(x, weight, alpha, out_dtype=torch.bfloat16)
    lowrank_add(y, x, stack, index, out=y)        # index: which adapter each token uses, or -1

Under autograd use apply_linear and apply_adapted (module.OPQLinear and module.AdaptedLinear
do); the other calls refuse tensors that require grad, as attention's do.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import attention, opq
from .opq import OPQ_BF16, OPQ_F32, _check

_P, _I, _L, _F, _Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t)

# signatures in header order
_SIGNATURES = {
    "opq_lowrank_workspace_bytes": (_Z, [_L, _L, _L, _L]),
    "opq_lowrank_add": (_I, [_P, _P, _L, _P, _L, _P, _L, _I, _P, _L, _I, _P, _Z, _P]),
    "opq_lowrank_backward_workspace_bytes": (_Z, [_L, _L, _L, _L, _L]),
    "opq_lowrank_backward": (_I, [_P, _P, _L, _P, _L, _P, _L, _P, _L, _I, _P, _L, _P, _P, _I, _P, _Z, _P]),
    "opq_linear_backward_workspace_bytes": (_Z, [_L, _L, _L]),
    "opq_linear_backward_codes_workspace_bytes": (_Z, [_L, _L, _L]),
    "opq_linear_backward": (_I, [_P, _P, _P, _P, _L, _L, _L, _F, _P, _I, _P, _Z, _P]),
    "opq_linear_backward_bits": (_I, [_P, _P, _P, _P, _L, _L, _L, _I, _F, _P, _I, _P, _Z, _P]),
    "opq_linear_backward_grouped": (_I, [_P, _P, _P, _P, _L, _L, _L, _L, _F, _P, _I, _P, _Z, _P]),
}

MAX_TRAINED = 1024   # adapters of one backward pass
_FLOATS = (torch.float32, torch.bfloat16)
_ready: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """libopq.so with the adapters' signatures set; raises if it or the extension is missing."""
    global _ready
    if _ready is None:
        lib = attention.load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _ready = lib
    return _ready


def _calls():
    return attention._ext or attention._calls()


class Adapters(NamedTuple):
    """A stack of low-rank adapters of one projection [in -> out]: token t with adapter i gets
    scale[i] * up[i]^T (down[i] x_t) added.  The rank is a multiple of 8, up to 128 (smaller ranks:
    rows of zeros); in and out are multiples of 8."""
    down: torch.Tensor    # bfloat16 [adapters, rank, in]
    up: torch.Tensor      # bfloat16 [adapters, rank, out]: the transpose of a layer's [out, rank]
    scale: torch.Tensor   # float32 [adapters]


def _float(what: str, dtype: torch.dtype) -> bool:
    if dtype not in _FLOATS:
        raise ValueError(f"{what} must be float32 or bfloat16, got {dtype}")
    return dtype == torch.bfloat16


def lowrank_add(y: Optional[torch.Tensor], x: torch.Tensor, adapters: Adapters, index: torch.Tensor,
                out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [tokens, out] (float32 or bfloat16; None: zeros) plus, for every token, its adapter's
    output.  x: bfloat16 [tokens, in]; index: int32 [tokens], the adapter of each token (outside
    0..adapters-1, such as -1: none, the token keeps its y).  Rows are dense, their strides free
    (multiples of 8).  Returns `out` (which may be y), or a new tensor of out_dtype (y's type
    by default, bfloat16 without y)."""
    if out_dtype is None:
        out_dtype = y.dtype if isinstance(y, torch.Tensor) else torch.bfloat16
    bf16 = _float("out_dtype", out_dtype) if out is None else False
    return _calls().lowrank_add(y, x, adapters, index, out, bf16, workspace)


def lowrank_backward(dy: torch.Tensor, x: torch.Tensor, adapters: Adapters, index: torch.Tensor,
                     dx: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     dx_dtype: torch.dtype = torch.bfloat16, grad_dtype: torch.dtype = torch.float32,
                     input_grad: bool = True, adapter_grads: bool = True,
                     workspace: Optional[torch.Tensor] = None
                     ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, d_down, d_up) from dy, bfloat16 [tokens, out].  dx: what the adapters give is added
    to `dx` [tokens, in] (None: zeros) in its type (dx_dtype without one), into `out` (which may be
    `dx`) or a new tensor.  d_down and d_up have the stack's shapes, in grad_dtype; adapters without
    tokens get zeros.  input_grad, adapter_grads: which are wanted (None in the place of others)."""
    return _calls().lowrank_backward(dy, x, adapters, index, dx, out, _float("dx_dtype", dx_dtype),
                                     _float("grad_dtype", grad_dtype), input_grad, adapter_grads, workspace)


# ------------------------------------------------------- through the projection

# what one call of the library takes; more tokens or weight rows go to it in blocks
_TOKENS, _ROWS = 1 << 22, 1 << 16


def linear_backward_workspace_bytes(m: int, n: int, k: int, bits: Optional[int] = None) -> int:
    """Workspace bytes of linear_backward (its largest block's): enough for codes of any width, or of
    `bits` bits, 4 of which need less."""
    ask = load().opq_linear_backward_codes_workspace_bytes if bits == 4 else load().opq_linear_backward_workspace_bytes
    if m <= _TOKENS and n <= _ROWS:
        return ask(m, n, k)
    sizes = [(a, b) for a in {min(m, _TOKENS), m % _TOKENS if m > _TOKENS else 0}
             for b in {min(n, _ROWS), n % _ROWS if n > _ROWS else 0}]
    return max(ask(a, b, k) for a, b in sizes)


def _check_rows(qw, n: int, k: int) -> None:
    for name, t in (("packed", qw.packed), ("sign", qw.sign)):
        opq._need_cuda(name, t, torch.int32, 2)
    opq._need_cuda("scale", qw.scale, torch.float32, 1)
    if tuple(qw.packed.shape) != (n, k // 8) or tuple(qw.sign.shape) != (n, k // 32) or tuple(qw.scale.shape) != (n,):
        raise ValueError(f"weight buffers do not match n={n}, k={k}")


def _backward_call(name, dy, weight, alpha, out, k, workspace, room) -> None:
    """One call of the library, its tensors checked, on their device."""
    m, n = dy.shape
    _check(name, getattr(load(), name)(
        dy.data_ptr(), weight[0].data_ptr(), weight[1].data_ptr(), weight[2].data_ptr(), m, n, k, *weight[3:], alpha,
        out.data_ptr(), OPQ_BF16 if out.dtype == torch.bfloat16 else OPQ_F32, opq._ptr(workspace), room,
        opq._stream(dy.device)))


def _backward_blocks(name, dy, weight, alpha, out, k, *space) -> None:
    """The call of more tokens or rows than the library takes at once."""
    m, n = dy.shape
    for t in range(0, m, _TOKENS):
        some, to = dy[t:t + _TOKENS], out[t:t + _TOKENS]
        if n <= _ROWS:
            _backward_call(name, some, weight, alpha, to, k, *space)
            continue
        total = to if to.dtype == torch.float32 else torch.empty(to.shape, device=dy.device)
        part = torch.empty_like(total)
        for r in range(0, n, _ROWS):
            block = type(weight)(*(w[r:r + _ROWS] for w in weight[:3]), *weight[3:])
            _backward_call(name, some[:, r:r + _ROWS].contiguous(), block, alpha, part if r else total, k, *space)
            if r:
                total.add_(part)
        if total is not to:
            to.copy_(total)


def linear_backward(dy: torch.Tensor, weight, alpha: float, out: Optional[torch.Tensor] = None,
                    out_dtype: torch.dtype = torch.bfloat16,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx [m, k] = dy [m, n] W', the gradient of opq.linear's x: dy bfloat16, weight any of
    opq's stored forms.  `workspace`: a device tensor of linear_backward_workspace_bytes(m, n, k,
    bits) bytes (by default one of torch's allocator).  More than 65536 weight rows (a vocabulary's) are
    taken in blocks, whose float32 sums are added in order."""
    opq._need_cuda("dy", dy, torch.bfloat16, 2)
    if torch.is_grad_enabled() and dy.requires_grad:
        raise RuntimeError("dy requires grad, which this call does not follow: detach it, or call under "
                           "torch.no_grad()")
    m = dy.shape[0]
    n, k = weight.shape
    if dy.shape[1] != n:
        raise ValueError(f"dy has n={dy.shape[1]}, weight has n={n}")
    given = out is not None
    if not given:
        _float("out_dtype", out_dtype)
        out = torch.empty((m, k), dtype=out_dtype, device=dy.device)
    else:
        opq._need_cuda("out", out, out.dtype, 2)
        _float("out", out.dtype)
        if tuple(out.shape) != (m, k):
            raise ValueError(f"out must have shape {(m, k)}, got {tuple(out.shape)}")
        if torch.is_grad_enabled() and out.requires_grad:
            raise RuntimeError("out requires grad, which this call does not follow")
        near = out.data_ptr() - dy.data_ptr()
        if out.numel() and dy.numel() and -out.numel() * out.element_size() < near < dy.numel() * 2:
            raise ValueError("out must not share memory with dy")
    for name, t in (("out", out), ("packed", weight.packed), ("sign", weight.sign), ("scale", weight[2])):
        if t.device != dy.device:
            raise ValueError(f"{name} must be on {dy.device}, got {t.device}")
    name, bits = "opq_linear_backward", 4
    if isinstance(weight, opq.BitsWeight):
        opq._check_bits(weight, n, k)
        name, bits = "opq_linear_backward_bits", weight.bits
    elif isinstance(weight, opq.GroupedWeight):
        opq._check_grouped(weight, n, k)
        name = "opq_linear_backward_grouped"
    else:
        _check_rows(weight, n, k)
    need = linear_backward_workspace_bytes(m, n, k, bits)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    elif workspace.device != dy.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dy.device}")
    room = 0 if workspace is None else workspace.numel() * workspace.element_size()
    call = _backward_call if m <= _TOKENS and n <= _ROWS else _backward_blocks
    with torch.cuda.device(dy.device):
        call(name, dy, weight, alpha, out, k, workspace, room)
    if given and not out.is_inference():   # written, so autograd learns of it
        torch.autograd.graph.increment_version(out)
    return out


# ------------------------------------------------------- the layers' projection

def project(x: torch.Tensor, weight, alpha: float, bias: Optional[torch.Tensor], out_dtype: torch.dtype) -> torch.Tensor:
    """opq.linear of x [m, k] (bfloat16) on x's device, with a workspace of the call's own: a layer may run
    on several streams at once."""
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        with torch.cuda.device(x.device):
            return opq.linear(x, weight, alpha, bias, None, opq.own_workspace, out_dtype)
    return opq.linear(x, weight, alpha, bias, None, opq.own_workspace, out_dtype)


# ------------------------------------------------------------------ autograd

def _dy(dy: torch.Tensor) -> torch.Tensor:
    """The gradient as the kernels take it: dense, from a 16-byte boundary on (a part of a longer
    gradient may start anywhere), in bfloat16, the type these layers' activations are rounded to on
    their way in."""
    dy = dy.to(torch.bfloat16).contiguous()
    return dy if dy.data_ptr() % 16 == 0 else dy.clone()


def _watched(weight):
    """A weight's tensors that autograd can watch for changes: those of inference mode have no
    version, and cannot be saved."""
    return [t for t in weight[:3] if not t.is_inference()]


class _Linear(torch.autograd.Function):
    """opq.linear; the weights are stored codes and take no gradient, so nothing of x is kept."""

    @staticmethod
    def forward(ctx, x, weight, alpha, bias, out_dtype):
        ctx.save_for_backward(*_watched(weight))
        ctx.how = (weight, alpha, x.dtype)
        return project(x.to(torch.bfloat16).contiguous(), weight, alpha, bias, out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        weight, alpha, dtype = ctx.how
        ctx.saved_tensors   # raises if the weight was changed
        dx = linear_backward(_dy(dy), weight, alpha, out_dtype=dtype)
        return dx, None, None, None, None


class _Adapted(torch.autograd.Function):
    """opq.linear with every token's adapter added: one output, written once more in place."""

    @staticmethod
    def forward(ctx, x, weight, alpha, bias, down, up, scale, index, out_dtype):
        xb = x.to(torch.bfloat16).contiguous()
        y = project(xb, weight, alpha, bias, out_dtype)
        lowrank_add(y, xb, Adapters(down, up, scale), index, out=y)
        ctx.save_for_backward(xb, down, up, scale, index, *_watched(weight))
        ctx.how = (weight, alpha, x.dtype)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        xb, down, up, scale, index = ctx.saved_tensors[:5]
        weight, alpha, dtype = ctx.how
        dy, dx = _dy(dy), None
        wants_x, wants = ctx.needs_input_grad[0], ctx.needs_input_grad[4] or ctx.needs_input_grad[5]
        if wants_x:
            dx = linear_backward(dy, weight, alpha, out_dtype=dtype)
        _, d_down, d_up = lowrank_backward(dy, xb, Adapters(down, up, scale), index, dx=dx, out=dx, grad_dtype=down.dtype,
                                           input_grad=wants_x, adapter_grads=wants)
        return dx, None, None, None, d_down, d_up, None, None, None


def apply_linear(x: torch.Tensor, weight, alpha: float, bias: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """opq.linear(x [m, k], float32 or bfloat16) that autograd differentiates with respect to x (not
    to the stored weights, nor to a bias).  The result has x's type unless out_dtype says otherwise;
    gradients of gradients are refused."""
    if bias is not None and bias.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("bias requires grad, which apply_linear does not follow: detach it")
    return _Linear.apply(x, weight, alpha, bias, out_dtype or x.dtype)


def apply_adapted(x: torch.Tensor, weight, alpha: float, bias: Optional[torch.Tensor], adapters: Adapters,
                  index: torch.Tensor, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """opq.linear of x [m, k] plus every token's adapter (lowrank_add), differentiated with respect
    to x, adapters.down and adapters.up (not to scale or bias).  Training a stack updates the
    adapters that `index` names and gives zeros for the others.  Gradients of gradients are refused."""
    for name, t in (("scale", adapters.scale), ("bias", bias)):
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{name} requires grad, which apply_adapted does not follow: detach it")
    if adapters.down.shape[0] > MAX_TRAINED and torch.is_grad_enabled() and any(
            t.requires_grad for t in (x, adapters.down, adapters.up)):
        raise ValueError(f"a backward pass takes up to {MAX_TRAINED} adapters, got {adapters.down.shape[0]}")
    return _Adapted.apply(x, weight, alpha, bias, adapters.down, adapters.up, adapters.scale, index, out_dtype or x.dtype)
