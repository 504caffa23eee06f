"""CPU tests of the attention side: its oracle pinned by closed forms, and the
library's host parts (frequencies, argument checks, exported symbols), which reach no
kernel launch."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import attention_oracle as AO
from w4a16_linear_amd import attention as A
from w4a16_linear_amd import opq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "opq_attention.h")
OK, NULL, SHAPE, ALPHA, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED, HIP = range(9)
FAKE = 0x7F0000000000          # an aligned, never dereferenced address
ODD = FAKE + 2


# ------------------------------------------------------------------ oracle

def test_e4m3_rounding_equals_torch_for_every_neighbourhood():
    """All 127 magnitudes, the midpoints between them and points just off them."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mid = (codes[1:] + codes[:-1]) / 2
    pts = np.concatenate([codes, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)])
    pts = np.concatenate([pts, -pts])
    ref = torch.from_numpy(pts).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(AO.round_e4m3(pts.astype(np.float32).astype(np.float64)), ref)


def test_cache_rows_by_hand():
    row = np.zeros((1, 64), np.float32)
    row[0, :3] = [448.0, -1.0, 0.0625]
    codes, scale = AO.cache_rows(row, "fp8")
    assert scale[0] == 1.0 and list(codes[0, :4]) == [448.0, -1.0, 0.0625, 0.0]
    codes, scale = AO.cache_rows(row, "opq4", alpha=1.0)   # uniform: 15 |x| / 448
    assert scale[0] == 448.0 and list(codes[0, :3]) == [1.0, 0.0, 0.0]
    codes, scale = AO.cache_rows(row, "bf16")
    assert scale[0] == 1.0 and list(codes[0, :3]) == [448.0, -1.0, 0.0625]
    for fmt in ("bf16", "fp8", "opq4"):
        for bad in (np.nan, np.inf, -np.inf):
            row[0, 5] = bad
            codes, scale = AO.cache_rows(row, fmt)
            assert np.isnan(scale[0]) and not codes.any()
        assert np.isnan(AO.cache_values(codes, scale)).all()
        tiny = np.full((1, 64), 2.0 ** -101, np.float32)
        codes, scale = AO.cache_rows(tiny, fmt)
        assert (scale[0] == 0.0 and not codes.any()) if fmt != "bf16" else codes[0, 0] == 2.0 ** -101


def test_rotary_oracle_is_a_turn():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 16))
    angle = rng.uniform(0, 6, (40, 4))
    table = np.stack([np.cos(angle), np.sin(angle)], -1)
    pos = rng.integers(0, 40, (3, 2))
    for layout in ("half", "interleaved"):
        y, _ = AO.rotary(x, pos, table, layout, (1, 3))
        assert np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        back, _ = AO.rotary(y, pos, table, layout, (1, 3), backward=True)
        assert np.allclose(back, x)
        z = np.exp(1j * angle[pos[1, 1], 2])   # pair 2 belongs to axis 1
        a, b = (2, 6) if layout == "half" else (4, 5)
        turned = (x[1, 0, a] + 1j * x[1, 0, b]) * z
        assert np.allclose([y[1, 0, a], y[1, 0, b]], [turned.real, turned.imag])


def test_attention_oracle_equals_torch():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, 2, 8), (9, 8), (9, 8)))
    seen = np.tril(np.ones((4, 4), bool))
    out, lse, spread, reach = AO.attention(q.numpy(), k.numpy(), v.numpy(), 5, seen, 0.3)
    for t in range(4):
        w = 0.3 * q[t] @ k[:6 + t].T
        assert np.allclose(out[t], (torch.softmax(w, -1) @ v[:6 + t]).numpy())
        assert np.allclose(lse[t], torch.logsumexp(w, -1).numpy())
    out, lse, _, _ = AO.attention(q.numpy(), k.numpy(), v.numpy(), 0, np.zeros((4, 4), bool), 0.3)
    assert not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("plant", ["half_up", "scale_127", "mask_shift", "turn_sign"])
def test_planted_mistakes_show(plant, monkeypatch):
    """The checks above are sharp: each planted mistake in the oracle changes what it gives."""
    rng = np.random.default_rng(5)
    if plant == "half_up":
        r = np.array([1.0625, 1.1875, 17.0])      # ties: to 1.0, 1.25, 16
        assert list(AO.round_e4m3(r)) == [1.0, 1.25, 16.0]
        step = np.array([0.125, 0.125, 2.0])
        assert list(np.floor(r / step + 0.5) * step) != [1.0, 1.25, 16.0]
    elif plant == "scale_127":
        x = rng.standard_normal((4, 64)).astype(np.float32)
        codes, scale = AO.cache_rows(x, "fp8")
        assert np.abs(codes).max(-1).min() == 448.0
    elif plant == "mask_shift":
        q, k = rng.standard_normal((3, 1, 8)), rng.standard_normal((5, 8))
        seen = np.tril(np.ones((3, 3), bool))
        a = AO.attention(q, k, k, 2, seen, 1.0)[0]
        assert not np.allclose(a, AO.attention(q, k, k, 2, np.roll(seen, 1, 1), 1.0)[0])
    else:
        x, pos = rng.standard_normal((2, 1, 8)), np.array([[3], [4]])
        t = np.stack([np.cos(np.arange(20).reshape(5, 4)), np.sin(np.arange(20).reshape(5, 4))], -1)
        assert not np.allclose(AO.rotary(x, pos, t, "half", (4,))[0],
                               AO.rotary(x, pos, t, "half", (4,), backward=True)[0])


# --------------------------------------------------------------- host parts

@pytest.fixture(scope="module")
def lib():
    return A.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(opq_\w+)\s*\(", text))
    assert names == set(A._SIGNATURES)
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("kw", [
    {}, dict(base=1e6), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="yarn", factor=16.0, original_len=4096.0),
    dict(scaling="yarn", factor=1.0, original_len=100.0, beta_fast=8.0, beta_slow=0.0)])
def test_frequencies(rot, kw):
    got = A.rotary_frequencies(rot, **kw)
    f, amp = AO.rotary_frequencies(rot, **kw)
    # two pow / exp-log evaluations in double: a few ulps of the exponent's magnitude
    assert np.allclose(got.freq, f, rtol=1e-13, atol=0.0)
    assert abs(got.amplitude - amp) <= 1e-15 * abs(amp)
    if kw.get("scaling") == "yarn" and kw["factor"] > 1 and rot == 128:
        g, _ = AO.rotary_frequencies(rot)
        assert got.freq[0] == g[0] and np.isclose(got.freq[-1], g[-1] / kw["factor"])


def test_frequency_errors(lib):
    f, amp = np.zeros(64), np.zeros(1)

    def call(rot=64, base=1e4, scaling=0, factor=1.0, n=0.0, fast=32.0, slow=1.0, out=f.ctypes.data):
        return lib.opq_rotary_frequencies(rot, base, scaling, factor, n, fast, slow, out, amp.ctypes.data)

    assert call() == OK
    assert call(out=None) == NULL
    for rot in (0, -2, 3, 1026):
        assert call(rot=rot) == SHAPE
    for base in (1.0, 0.0, -1.0, math.inf, math.nan):
        assert call(base=base) == ALPHA
    for factor in (0.5, math.nan, math.inf):
        assert call(scaling=1, factor=factor) == ALPHA
        assert call(factor=factor) == OK              # not used
    assert call(scaling=3, factor=2.0) == ALPHA       # no original length
    assert call(scaling=3, factor=2.0, n=10.0, fast=1.0, slow=1.0) == ALPHA
    assert call(scaling=3, factor=2.0, n=10.0, slow=-1.0) == ALPHA
    assert call(scaling=4, factor=2.0) == DTYPE
    with pytest.raises(ValueError):
        A.rotary_frequencies(64, scaling="other")


def test_table_and_rotary_argument_checks(lib):
    t = lib.opq_rotary_table
    assert t(None, 8, 8, 1.0, FAKE, None) == NULL
    assert t(FAKE, 8, 8, 1.0, None, None) == NULL
    for pairs, n in ((0, 8), (513, 8), (8, -1)):
        assert t(FAKE, pairs, n, 1.0, FAKE, None) == SHAPE
    assert t(ODD, 8, 8, 1.0, FAKE, None) == ALIGN
    assert t(FAKE, 512, 1 << 31, 1.0, FAKE, None) == UNSUPPORTED
    assert t(FAKE, 8, 0, 1.0, None, None) == OK
    sec = (ctypes.c_int32 * 4)(8, 8, 8, 8)

    def call(x=FAKE, dtype=1, tokens=4, heads=2, dim=64, pos=FAKE, axes=1, s=(32,), table=FAKE, n=16,
             rot=64, layout=0, out=FAKE):
        sec = (ctypes.c_int32 * max(1, len(s)))(*s)
        return lib.opq_rotary(x, dtype, tokens, heads, dim, heads * dim, dim, pos, axes, sec, table, n,
                              rot, layout, 0, out, heads * dim, dim, None)

    for kw in (dict(x=None), dict(out=None), dict(pos=None), dict(table=None)):
        assert call(**kw) == NULL
    assert lib.opq_rotary(FAKE, 1, 4, 2, 64, 128, 64, FAKE, 1, None, FAKE, 16, 64, 0, 0, FAKE, 128, 64,
                          None) == NULL
    for kw in (dict(tokens=-1), dict(heads=-1), dict(dim=0), dict(rot=66), dict(rot=0), dict(rot=7, s=(3,)),
               dict(axes=0), dict(axes=5), dict(s=(31,)), dict(s=(0,)), dict(axes=2, s=(33, -1)), dict(n=-1),
               dict(dim=70000), dict(dim=2048, rot=2048, s=(1024,))):
        assert call(**kw) == SHAPE, kw
    assert call(x=FAKE + 1) == ALIGN
    assert call(dtype=0, x=ODD) == ALIGN               # float32 needs 4 bytes
    assert call(x=ODD, tokens=0) == OK                 # bfloat16 needs 2
    assert call(pos=ODD) == ALIGN and call(table=ODD) == ALIGN
    assert call(dtype=2) == DTYPE and call(layout=2) == DTYPE
    assert call(tokens=1 << 36, heads=16) == UNSUPPORTED
    assert call(heads=1 << 25) == UNSUPPORTED
    assert call(tokens=0) == OK and call(heads=0) == OK
    assert len(sec) == 4


def _cache(**kw):
    a = dict(k=FAKE, k_sign=None, k_scale=FAKE, v=FAKE, v_sign=None, v_scale=FAKE, pages=4, heads=2, page=16,
             dim=64, format=1, alpha=0.73)
    a.update(kw)
    return A._CCache(*(a[n] for n, _ in A._CCache._fields_))


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v_scale=None), NULL), (dict(format=2), NULL), (dict(format=2, k_sign=FAKE), NULL),
    (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=0), SHAPE), (dict(dim=96), SHAPE),
    (dict(heads=0), SHAPE), (dict(pages=-1), SHAPE),
    (dict(format=2, k_sign=FAKE, v_sign=FAKE, alpha=0.01), ALPHA),
    (dict(format=2, k_sign=FAKE, v_sign=FAKE, alpha=math.nan), ALPHA),
    (dict(k=ODD), ALIGN), (dict(v_scale=ODD), ALIGN), (dict(format=3), DTYPE), (dict(format=-1), DTYPE),
    (dict(pages=1 << 27), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_checks(lib, kw, status):
    c = _cache(**kw)
    ref = ctypes.byref(c)
    assert lib.opq_cache_write(ref, FAKE, 128, 64, FAKE, 128, 64, 1, 3, FAKE, None) == status
    assert lib.opq_cache_read(ref, 3, FAKE, FAKE, FAKE, 1, None) == status
    assert lib.opq_cache_attention(ref, FAKE, 1, 1, 4, 256, 256, 64, FAKE, 1 if status != UNSUPPORTED else 1,
                                   FAKE, None, 0, None, 0, 1.0, FAKE, None, None, 0, None) == status


def test_write_and_read_argument_checks(lib):
    c = _cache()
    ref = ctypes.byref(c)
    w = lib.opq_cache_write
    assert w(None, FAKE, 128, 64, FAKE, 128, 64, 1, 3, FAKE, None) == NULL
    assert w(ref, None, 128, 64, FAKE, 128, 64, 1, 3, FAKE, None) == NULL
    assert w(ref, FAKE, 128, 64, FAKE, 128, 64, 1, 3, None, None) == NULL
    assert w(ref, FAKE, 128, 64, FAKE, 128, 64, 1, -1, FAKE, None) == SHAPE
    assert w(ref, FAKE, 128, 64, FAKE + 1, 128, 64, 1, 3, FAKE, None) == ALIGN
    assert w(ref, FAKE, 128, 64, FAKE, 128, 64, 0, 3, ODD, None) == ALIGN
    assert w(ref, FAKE, 128, 64, FAKE, 128, 64, 2, 3, FAKE, None) == DTYPE
    assert w(ref, FAKE, 128, 64, FAKE, 128, 64, 1, 1 << 31, FAKE, None) == UNSUPPORTED
    assert w(ref, None, 128, 64, None, 128, 64, 1, 0, None, None) == OK
    r = lib.opq_cache_read
    assert r(ref, 3, FAKE, None, FAKE, 1, None) == NULL
    assert r(ref, 3, FAKE, ODD, FAKE, 1, None) == ALIGN
    assert r(ref, 3, FAKE, FAKE, FAKE, 7, None) == DTYPE
    assert r(ref, 0, None, None, None, 1, None) == OK


def test_move_argument_checks(lib):
    ref = ctypes.byref(_cache())
    m = lib.opq_cache_move
    assert m(None, 1, 1, FAKE, FAKE, None) == NULL and m(ref, 1, 1, None, FAKE, None) == NULL
    assert m(ref, -1, 1, FAKE, FAKE, None) == SHAPE and m(ref, 1, -1, FAKE, FAKE, None) == SHAPE
    assert m(ref, 1, 1, FAKE, ODD, None) == ALIGN
    for batch, count in ((65536, 1), (1, 129)):
        assert m(ref, batch, count, FAKE, FAKE, None) == UNSUPPORTED
    assert m(ref, 0, 1, None, None, None) == OK and m(ref, 1, 0, None, None, None) == OK
    for kw, status in BAD_CACHES:
        assert m(ctypes.byref(_cache(**kw)), 1, 1, FAKE, FAKE, None) == status


def test_attention_argument_checks(lib):
    c = _cache()

    def call(q=FAKE, batch=1, draft=2, heads=4, strides=(512, 256, 64), table=FAKE, max_pages=3, lens=FAKE,
             counts=None, max_len=8, mask=None, mb=0, scale=1.0, out=FAKE, lse=None, ws=None, wsb=0):
        return lib.opq_cache_attention(ctypes.byref(c), q, batch, draft, heads, *strides, table, max_pages, lens,
                                       counts, max_len, mask, mb, scale, out, lse, ws, wsb, None)

    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(batch=-1), dict(draft=-1), dict(heads=3), dict(heads=0), dict(max_pages=-1), dict(max_len=-1),
               dict(max_len=49), dict(mb=-1), dict(max_pages=1 << 28)):
        assert call(**kw) == SHAPE, kw
    for s in (math.nan, math.inf):
        assert call(scale=s) == ALPHA
    for kw in (dict(q=ODD), dict(lens=ODD), dict(counts=ODD), dict(mask=ODD), dict(lse=ODD), dict(out=ODD),
               dict(ws=ODD, wsb=1 << 20), dict(strides=(512, 257, 64)), dict(strides=(512, 256, 60))):
        assert call(**kw) == ALIGN, kw
    need = lib.opq_cache_attention_workspace_bytes(1, 2, 4, 2, 64, 100000)
    assert need > 0 and need % 256 == 0
    big = dict(max_pages=10000, max_len=100000)
    assert call(**big) == WORKSPACE
    assert call(**big, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert call(batch=70000) == UNSUPPORTED
    assert call(draft=1 << 17, max_len=0) == UNSUPPORTED
    assert call(batch=0) == OK and call(draft=0) == OK
    ws = lib.opq_cache_attention_workspace_bytes
    assert ws(0, 1, 4, 2, 64, 100) == 0 and ws(1, 1, 3, 2, 64, 100) == 0 and ws(1, 1, 4, 2, 65, 100) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(2, 2, 64)
    pos, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        A.rotary(x, pos, table)
    with pytest.raises(ValueError, match="layout"):
        A.rotary(x, pos, table, layout="third")
    cache = A.new_cache(2, 2, 16, 64, "fp8", device="cpu")
    assert (cache.pages, cache.heads, cache.page, cache.dim) == (2, 2, 16, 64)
    assert A.new_cache(2, 2, 16, 128, "opq4", device="cpu").dim == 128
    with pytest.raises(ValueError, match="CUDA"):
        A.cache_write(cache, x, x, pos)
    with pytest.raises(ValueError, match="CUDA"):
        A.cache_read(cache, pos)
    with pytest.raises(ValueError, match="CUDA"):
        A.tree_attention(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), cache, pos[None], pos[:1])
    for kw in (dict(fmt="int3"), dict(dim=80), dict(page=24)):
        with pytest.raises(ValueError):
            A.new_cache(**{**dict(pages=1, heads=1, page=16, dim=64, device="cpu"), **kw})


def test_tree_mask():
    parents = torch.tensor([[-1, 0, 0, 1, 2], [-1, -1, 1, 2, 3]], dtype=torch.int32)
    m = A.tree_mask(parents).numpy()[..., 0]
    assert list(m[0]) == [0b1, 0b11, 0b101, 0b1011, 0b10101]
    assert list(m[1]) == [0b1, 0b10, 0b110, 0b1110, 0b11110]
    chain = A.tree_mask(torch.arange(-1, 39, dtype=torch.int32)[None]).numpy().view(np.uint32)
    assert chain.shape == (1, 40, 2) and chain[0, 39, 0] == 0xFFFFFFFF and chain[0, 39, 1] == 0xFF
    for bad in ([[0]], [[-2]], [[-1, 1]]):
        with pytest.raises(ValueError):
            A.tree_mask(torch.tensor(bad, dtype=torch.int32))


def test_status_text_is_the_librarys(lib):
    with pytest.raises(opq.OpqError) as e:
        A.rotary_frequencies(3)
    assert e.value.status == SHAPE
