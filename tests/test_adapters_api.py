"""The adapters' C ABI and binding without a GPU: symbols, the order of the argument checks,
what is refused before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from w4a16_linear_amd import adapters as L
from w4a16_linear_amd import opq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "opq_adapters.h")
OK, NULL, SHAPE, ALPHA, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6, 7
FAKE, ODD = 1 << 20, (1 << 20) + 2     # never read: every call here ends before a launch


class Stack(ctypes.Structure):
    _fields_ = [("down", ctypes.c_void_p), ("up", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("rank", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64)]


def _stack(**kw):
    return Stack(**{**dict(down=FAKE, up=FAKE, scale=FAKE, count=2, rank=16, k=64, n=128), **kw})


@pytest.fixture(scope="module")
def lib():
    return L.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(opq_\w+)\s*\(", text))
    assert names == set(L._SIGNATURES)
    for n in names:
        assert hasattr(lib, n)


def test_status_codes_are_the_headers():
    text = open(os.path.join(ROOT, "include", "opq.h")).read()
    for name, value in (("NULL", NULL), ("SHAPE", SHAPE), ("ALPHA", ALPHA), ("ALIGN", ALIGN), ("DTYPE", DTYPE),
                        ("WORKSPACE", WORKSPACE), ("UNSUPPORTED", UNSUPPORTED)):
        assert re.search(rf"OPQ_ERR_{name}\s*=\s*{value}\b|#define OPQ_ERR_{name}\s+{value}\b", text), name


BAD_STACKS = [(dict(down=None), NULL), (dict(up=None), NULL), (dict(scale=None), NULL), (dict(rank=0), SHAPE),
              (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(k=0), SHAPE), (dict(k=60), SHAPE), (dict(n=4), SHAPE),
              (dict(n=129), SHAPE), (dict(count=-1), SHAPE), (dict(down=ODD), ALIGN), (dict(up=FAKE + 8), ALIGN),
              (dict(scale=ODD), ALIGN)]


def test_add_checks(lib):
    def call(a=None, x=FAKE, xs=64, index=FAKE, m=3, y=FAKE, ys=128, yd=1, out=FAKE, os_=128, od=1, ws=FAKE,
             wsb=1 << 30):
        return lib.opq_lowrank_add(ctypes.byref(a or _stack()), x, xs, index, m, y, ys, yd, out, os_, od, ws, wsb, None)

    assert lib.opq_lowrank_add(None, FAKE, 64, FAKE, 3, FAKE, 128, 1, FAKE, 128, 1, FAKE, 1 << 30, None) == NULL
    for kw, status in BAD_STACKS:
        assert call(_stack(**kw)) == status, kw
    for kw in (dict(x=None), dict(index=None), dict(out=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(m=-1), dict(xs=56), dict(xs=-64), dict(ys=120), dict(os_=0), dict(os_=120)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=ODD), dict(index=ODD), dict(y=ODD), dict(out=ODD), dict(ws=ODD), dict(xs=68), dict(ys=132),
               dict(os_=130)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(yd=2), dict(od=-1)):
        assert call(**kw) == DTYPE, kw
    need = lib.opq_lowrank_workspace_bytes(3, 64, 128, 16)
    assert need >= 3 * 16 * 4
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    for kw in (dict(m=(1 << 22) + 1), dict(m=1 << 22, xs=1 << 18), dict(m=1 << 22, ys=1 << 18), dict(m=1 << 22, os_=1 << 18)):
        assert call(**{**kw, "wsb": 1 << 62}) == UNSUPPORTED, kw
    assert call(_stack(k=(1 << 20) + 8), xs=(1 << 20) + 8) == UNSUPPORTED
    assert call(_stack(count=(1 << 30) + 1)) == UNSUPPORTED
    assert call(m=0, x=None, index=None, y=None, out=None, ws=None, wsb=0) == OK
    assert lib.opq_lowrank_workspace_bytes(-1, 64, 128, 16) == 0 and lib.opq_lowrank_workspace_bytes(3, 64, 128, 12) == 0


def test_backward_checks(lib):
    def call(a=None, dy=FAKE, dys=128, x=FAKE, xs=64, index=FAKE, m=3, dx=FAKE, dxs=64, dxd=1, out=FAKE, os_=64, dd=FAKE,
             du=FAKE, gd=0, ws=FAKE, wsb=1 << 40):
        return lib.opq_lowrank_backward(ctypes.byref(a or _stack()), dy, dys, x, xs, index, m, dx, dxs, dxd, out, os_, dd,
                                        du, gd, ws, wsb, None)

    for kw, status in BAD_STACKS:
        assert call(_stack(**kw)) == status, kw
    for kw in (dict(dy=None), dict(x=None), dict(index=None), dict(dd=None), dict(du=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(m=-1), dict(dys=120), dict(xs=56), dict(dxs=8), dict(os_=0)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(dy=ODD), dict(x=ODD), dict(index=ODD), dict(dx=ODD), dict(out=ODD), dict(dd=ODD), dict(du=ODD),
               dict(ws=ODD), dict(dys=132), dict(xs=70), dict(dxs=68), dict(os_=68)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(dxd=2), dict(gd=2)):
        assert call(**kw) == DTYPE, kw
    need = lib.opq_lowrank_backward_workspace_bytes(3, 64, 128, 16, 2)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE
    assert call(_stack(count=1025)) == UNSUPPORTED
    assert call(m=(1 << 22) + 1, wsb=1 << 62) == UNSUPPORTED
    assert call(out=None, dd=None, du=None) == OK
    assert call(_stack(count=0, down=None, up=None, scale=None), m=0, dy=None, x=None, index=None) == OK


def test_linear_backward_checks(lib):
    def call(fn="", dy=FAKE, packed=FAKE, sign=FAKE, scale=FAKE, m=4, n=64, k=256, extra=(), alpha=0.73, dx=FAKE, dd=1,
             ws=FAKE, wsb=1 << 40):
        return getattr(lib, "opq_linear_backward" + fn)(dy, packed, sign, scale, m, n, k, *extra, alpha, dx, dd, ws, wsb, None)

    for fn, extra in (("", ()), ("_bits", (5,)), ("_grouped", (128,))):
        for kw in (dict(dy=None), dict(packed=None), dict(sign=None), dict(scale=None), dict(dx=None)):
            assert call(fn, extra=extra, **kw) == NULL, kw
        for kw in (dict(m=-1), dict(n=-1), dict(k=250)):
            assert call(fn, extra=extra, **kw) == SHAPE, kw
        for a in (0.0, float("nan")):
            assert call(fn, extra=extra, alpha=a) == ALPHA
        for kw in (dict(dy=ODD), dict(packed=ODD), dict(sign=ODD), dict(scale=ODD), dict(dx=ODD), dict(ws=ODD)):
            assert call(fn, extra=extra, **kw) == ALIGN, kw
        assert call(fn, extra=extra, dd=3) == DTYPE
        need = lib.opq_linear_backward_workspace_bytes(4, 64, 256)
        assert call(fn, extra=extra, wsb=need - 1) == WORKSPACE
        for kw in (dict(n=65568), dict(k=65536 + 256), dict(m=(1 << 22) + 1)):
            assert call(fn, extra=extra, **kw) == UNSUPPORTED, kw
        assert call(fn, extra=extra, m=0, dy=None, dx=None, ws=None, wsb=0) == OK
    assert call("_bits", extra=(7,)) == SHAPE and call("_grouped", extra=(48,)) == SHAPE


def test_binding_refuses_what_it_cannot_pass_on():
    a = L.Adapters(torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 32, dtype=torch.bfloat16), torch.ones(2))
    x, y, index = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.lowrank_add(y, x, a, index)
    with pytest.raises(ValueError, match="CUDA"):
        L.lowrank_backward(y, x, a, index)
    with pytest.raises(ValueError, match="out_dtype"):
        L.lowrank_add(y, x, a, index, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="grad_dtype"):
        L.lowrank_backward(y, x, a, index, grad_dtype=torch.float64)
    w = opq.QuantizedWeight(torch.zeros(32, 8, dtype=torch.int32), torch.zeros(32, 2, dtype=torch.int32), torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        L.linear_backward(torch.zeros(3, 32, dtype=torch.bfloat16), w, 0.73)


def test_in_place_means_the_same_rows(lib):
    """y as out (dx as dx_out) with another stride or type would leave rows without an adapter unwritten."""
    def add(m, ys, yd, od, out=FAKE):
        return lib.opq_lowrank_add(ctypes.byref(_stack()), FAKE, 64, FAKE, m, FAKE, ys, yd, out, 128, od, FAKE, 1 << 40, None)

    assert add(3, 136, 1, 1) == UNSUPPORTED and add(3, 128, 0, 1) == UNSUPPORTED and add(1, 128, 1, 0) == UNSUPPORTED
    assert lib.opq_lowrank_backward(ctypes.byref(_stack()), FAKE, 128, FAKE, 64, FAKE, 3, FAKE, 72, 1, FAKE, 64, FAKE, FAKE, 0,
                                    FAKE, 1 << 40, None) == UNSUPPORTED


def test_what_4_bit_codes_need(lib):
    """W' is written for longer calls only, and once: what few tokens need are their split sums."""
    every, codes = lib.opq_linear_backward_workspace_bytes, lib.opq_linear_backward_codes_workspace_bytes
    for m in (1, 8, 64, 65, 333, 512):
        for n, k in ((3840, 3840), (20480, 3840), (3840, 10240), (65536, 65536), (1000, 96)):
            # at most 512 workgroups' planes, 128 columns each; dy with longer rows; whole MiB
            assert codes(m, n, k) <= 512 * m * 128 * 4 + 2 * m * (n + 63) + (2 << 20), (m, n, k)
    for m in (513, 4096):
        for n, k in ((3840, 3840), (20480, 3840), (1001, 96)):
            assert codes(m, n, k) >= n * k * 2 and every(m, n, k) >= codes(m, n, k) + n * k * 2 - (1 << 20)
    for size in ((0, 64, 64), (4, 65537, 64), (4, 64, 65568), ((1 << 22) + 1, 64, 64), (4, 64, 40)):
        assert every(*size) == codes(*size) == 0

    def call(fn, m, n, k, wsb, extra=()):
        return getattr(lib, "opq_linear_backward" + fn)(FAKE, FAKE, FAKE, FAKE, m, n, k, *extra, 0.73, FAKE, 1, FAKE, wsb, None)

    for m, n, k in ((8, 20480, 3840), (600, 3840, 512)):
        for fn, extra, need in (("", (), codes), ("_bits", (4,), codes), ("_grouped", (128,), codes), ("_bits", (5,), every)):
            assert call(fn, m, n, k, need(m, n, k) - 1, extra) == WORKSPACE
