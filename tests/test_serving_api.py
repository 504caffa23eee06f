"""Argument checks of the pages' and the verification's C calls, without a GPU: every call here
ends before a launch."""
import ctypes

import pytest
import torch

from w4a16_linear_amd import attention as A

OK, NULL, SHAPE, ALPHA, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6, 7
FAKE, ODD = 1 << 20, (1 << 20) + 2


@pytest.fixture(scope="module")
def lib():
    return A.load()


def test_resize_checks(lib):
    def call(table=FAKE, lens=FAKE, rows=3, columns=4, pages=9, page=16, out=FAKE, missing=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.opq_pages_resize(table, lens, rows, columns, pages, page, out, missing, ws, wsb, None)

    for kw in (dict(table=None), dict(lens=None), dict(out=None), dict(missing=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(rows=-1), dict(columns=-1), dict(pages=0), dict(page=8), dict(page=24), dict(page=0)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(table=ODD), dict(lens=ODD), dict(out=ODD), dict(missing=ODD), dict(ws=FAKE + 8)):
        assert call(**kw) == ALIGN, kw
    need = lib.opq_pages_workspace_bytes(3, 9)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    for kw in (dict(rows=(1 << 20) + 1), dict(pages=(1 << 20) + 1), dict(rows=1 << 10, columns=(1 << 18) + 1), dict(page=1 << 31)):
        assert call(**kw) == UNSUPPORTED, kw
    ws = lib.opq_pages_workspace_bytes
    assert ws(-1, 9) == 0 and ws(3, 0) == 0 and ws(0, 1) > 0 and ws(1 << 20, 1 << 20) > 0


def test_fork_checks(lib):
    def call(table=FAKE, lens=FAKE, rows=3, columns=4, parents=FAKE, new=5, pages=9, page=16, out=FAKE, out_lens=FAKE, src=FAKE,
             dst=FAKE, missing=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.opq_pages_fork(table, lens, rows, columns, parents, new, pages, page, out, out_lens, src, dst, missing, ws,
                                  wsb, None)

    for name in ("table", "lens", "parents", "out", "out_lens", "src", "dst", "missing"):
        assert call(**{name: None}) == NULL and call(**{name: ODD}) == ALIGN, name
    for kw in (dict(rows=-1), dict(new=-1), dict(columns=-1), dict(pages=0), dict(page=17)):
        assert call(**kw) == SHAPE, kw
    assert call(wsb=lib.opq_pages_workspace_bytes(5, 9) - 1) == WORKSPACE
    for kw in (dict(rows=(1 << 20) + 1), dict(new=(1 << 20) + 1), dict(new=1 << 11, columns=(1 << 17) + 1)):
        assert call(**kw) == UNSUPPORTED, kw


def test_compact_checks(lib):
    def call(table=FAKE, rows=3, columns=4, pages=9, out=FAKE, src=FAKE, dst=FAKE, used=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.opq_pages_compact(table, rows, columns, pages, out, src, dst, used, ws, wsb, None)

    for name in ("table", "out", "src", "dst", "used"):
        assert call(**{name: None}) == NULL and call(**{name: ODD}) == ALIGN, name
    for kw in (dict(rows=-1), dict(columns=-1), dict(pages=0)):
        assert call(**kw) == SHAPE, kw
    assert call(wsb=8) == WORKSPACE and call(pages=(1 << 20) + 1) == UNSUPPORTED


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_sign", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_sign", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("dim", ctypes.c_int64), ("format", ctypes.c_int), ("alpha", ctypes.c_float)]


def _cache(**kw):
    return Cache(**{**dict(k=FAKE, k_sign=FAKE, k_scale=FAKE, v=FAKE, v_sign=FAKE, v_scale=FAKE, pages=3, heads=2, page=16, dim=64,
                           format=2, alpha=0.73), **kw})


def test_copy_checks(lib):
    c = lib.opq_cache_copy_pages
    ref = ctypes.byref(_cache())
    assert c(None, 1, FAKE, FAKE, None) == NULL and c(ref, 1, None, FAKE, None) == NULL and c(ref, 1, FAKE, None, None) == NULL
    assert c(ref, -1, FAKE, FAKE, None) == SHAPE and c(ref, 1, ODD, FAKE, None) == ALIGN
    assert c(ref, (1 << 20) + 1, FAKE, FAKE, None) == UNSUPPORTED and c(ref, 0, None, None, None) == OK
    for kw, status in ((dict(k=None), NULL), (dict(v_sign=None), NULL), (dict(page=8), SHAPE), (dict(dim=80), SHAPE),
                       (dict(alpha=0.0), ALPHA), (dict(v_scale=ODD), ALIGN), (dict(format=7), DTYPE),
                       (dict(pages=1 << 28), UNSUPPORTED)):
        assert c(ctypes.byref(_cache(**kw)), 1, FAKE, FAKE, None) == status, kw


def test_verify_checks(lib):
    def call(p=FAKE, dtype=0, batch=2, draft=3, vocab=100, bs=300, ts=100, tokens=FAKE, u=FAKE, q=None, qb=200, qt=100,
             parents=None, counts=None, kept=FAKE, count=FAKE, nxt=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.opq_verify_drafts(p, dtype, batch, draft, vocab, bs, ts, tokens, u, q, qb, qt, parents, counts, kept, count,
                                     nxt, ws, wsb, None)

    for name in ("p", "tokens", "u", "kept", "count", "nxt"):
        assert call(**{name: None}) == NULL and call(**{name: ODD}) == ALIGN, name
    for name in ("q", "parents", "counts"):
        assert call(**{name: ODD}) == ALIGN, name
    assert call(p=FAKE + 1, dtype=1) == ALIGN and call(dtype=2) == DTYPE
    for kw in (dict(batch=-1), dict(draft=0), dict(vocab=0), dict(bs=-1), dict(ts=-1), dict(q=FAKE, qb=-1), dict(q=FAKE, qt=-1)):
        assert call(**kw) == SHAPE, kw
    need = lib.opq_verify_drafts_workspace_bytes(2, 100)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    for kw in (dict(batch=65536), dict(draft=1025), dict(vocab=(1 << 22) + 1), dict(q=FAKE, parents=FAKE), dict(bs=1 << 39),
               dict(ts=1 << 38), dict(q=FAKE, qb=1 << 39)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(batch=0, p=None, tokens=None, u=None, kept=None, count=None, nxt=None, ws=None, wsb=0) == OK


def test_binding_refuses_host_tensors():
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: A.pages_resize(t, n, 9, 16), lambda: A.pages_fork(t, n, n, 9, 16), lambda: A.pages_compact(t, 9),
                 lambda: A.cache_copy_pages(A.new_cache(2, 1, 16, 64, device="cpu"), n, n),
                 lambda: A.verify_drafts(torch.zeros(2, 3, 9), t, torch.zeros(2, 3))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
