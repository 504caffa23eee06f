"""Rotary positions on the GPU against the float64 oracle: both layouts, parts of the
head, several axes, strides and alignments, in place, the backward pass."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as AO
from w4a16_linear_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32, UBF = 2.0 ** -24, 2.0 ** -8   # half an ulp of 1 in float32 and bfloat16


def _table(rng, length, pairs):
    angle = rng.uniform(-9, 9, (length, pairs))
    return np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


def _check(got, x, pos, table, layout, sections, backward=False):
    ref, mag = AO.rotary(x.double().cpu().numpy(), pos, table, layout, sections, backward)
    # two products and a sum in float32 (the sum may be fused), then the result's type
    bound = 3 * U32 * mag + (UBF * (np.abs(ref) + 3 * U32 * mag) if got.dtype == torch.bfloat16 else 0) + 1e-44
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= bound).all(), float((err - bound).max())


CASES = [  # tokens, heads, dim, rot, sections
    (1, 1, 64, 64, None), (3, 5, 128, 128, None), (70, 7, 128, 64, None), (5, 3, 80, 80, None),
    (4, 2, 96, 24, None), (33, 40, 128, 128, (16, 24, 24)), (9, 3, 64, 48, (6, 9, 9)), (2, 3, 65, 6, None),
    (3, 2, 7, 2, None), (6, 2, 256, 254, (100, 7, 19, 1)), (700, 16, 128, 128, None), (130, 130, 96, 32, (8, 8))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot,sections", CASES)
def test_against_oracle(gpu_lib, tokens, heads, dim, rot, sections, layout, dtype):
    rng = np.random.default_rng(tokens * 131 + dim)
    table = _table(rng, 50, rot // 2)
    sections = sections or (rot // 2,)
    pos = rng.integers(0, 50, (tokens, len(sections))).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DEV, dtype)
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    _check(A.rotary(x, p, t, layout, sections), x, pos, table, layout, sections)
    _check(A.rotary_backward(x, p, t, layout, sections), x, pos, table, layout, sections, True)
    keep = x.clone()
    assert A.rotary(x, p, t, layout, sections, out=x) is x
    _check(x, keep, pos, table, layout, sections)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,token_pad,head_pad", [(0, 0, 0), (1, 0, 0), (8, 3, 0), (4, 0, 5), (16, 8, 8)])
def test_strides_and_alignment(gpu_lib, layout, dtype, offset, token_pad, head_pad):
    """Rows cut from a wider buffer, at any element: what lies between them stays."""
    tokens, heads, dim = 11, 6, 64
    rng = np.random.default_rng(offset + 10 * token_pad + head_pad)
    table = _table(rng, 20, 32)
    pos = rng.integers(0, 20, (tokens, 1)).astype(np.int32)
    hs = dim + head_pad
    ts = heads * hs + token_pad
    flat = torch.from_numpy(rng.standard_normal(offset + tokens * ts).astype(np.float32)).to(DEV, dtype)
    view = flat[offset:].as_strided((tokens, heads, dim), (ts, hs, 1))
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    _check(A.rotary(view, p, t, layout), view, pos, table, layout, (32,))
    before, inner = flat.clone(), torch.zeros(flat.shape, dtype=torch.bool, device=DEV)
    inner[offset:].as_strided((tokens, heads, dim), (ts, hs, 1))[:] = True
    A.rotary(view, p, t, layout, out=view)
    assert torch.equal(flat[~inner], before[~inner])
    _check(view, before[offset:].as_strided((tokens, heads, dim), (ts, hs, 1)), pos, table, layout, (32,))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1])
def test_large_calls(gpu_lib, layout, dtype, offset):
    """Enough work for several heads a thread, a number of heads that is no multiple of
    theirs, a part of the head that is copied; aligned and not, apart and in place."""
    tokens, heads, dim, rot = 601, 53, 128, 64
    rng = np.random.default_rng(7 + offset)
    table = _table(rng, 40, rot // 2)
    pos = rng.integers(0, 40, (tokens, 1)).astype(np.int32)
    flat = torch.from_numpy(rng.standard_normal(offset + tokens * heads * dim).astype(np.float32)).to(DEV, dtype)
    x = flat[offset:].view(tokens, heads, dim)
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    y = A.rotary(x, p, t, layout)
    _check(y, x, pos, table, layout, (rot // 2,))
    A.rotary(x, p, t, layout, out=x)
    assert torch.equal(x, y)


def test_positions_that_start_inside_an_array(gpu_lib):
    table = torch.from_numpy(_table(np.random.default_rng(3), 30, 32)).to(DEV)
    pos = torch.arange(29, -1, -1, dtype=torch.int32, device=DEV)
    x = torch.randn(30, 2, 64, device=DEV)
    assert torch.equal(A.rotary(x[3:], pos[3:], table), A.rotary(x, pos, table)[3:])


def test_broadcast_head(gpu_lib):
    """A head seen by all (stride 0) is read once per head; its gradient is the sum."""
    rng = np.random.default_rng(4)
    table = _table(rng, 20, 32)
    pos = rng.integers(0, 20, (5, 1)).astype(np.int32)
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    one = torch.randn(5, 1, 64, device=DEV, requires_grad=True)
    y = A.apply_rotary(one.expand(5, 3, 64), p, t)
    g = torch.randn(5, 3, 64, device=DEV)
    (y * g).sum().backward()
    ref, mag = AO.rotary(g.double().cpu().numpy(), pos, table, "half", (32,), backward=True)
    err = np.abs(one.grad.double().cpu().numpy()[:, 0] - ref.sum(1))
    assert (err <= 6 * U32 * mag.sum(1)).all()   # three roundings each, two more of the sum


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(gpu_lib, layout):
    """The turn is linear, so a difference of outputs has no truncation error, only the
    float32 rounding of both outputs."""
    rng = np.random.default_rng(6)
    tokens, heads, dim, sections = 4, 2, 16, (2, 4)
    table = _table(rng, 20, 6)
    pos = rng.integers(0, 20, (tokens, 2)).astype(np.int32)
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    x = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DEV).requires_grad_()
    w = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DEV)
    (A.apply_rotary(x, p, t, layout, sections) * w).sum().backward()
    h = 0.5
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 7), (3, 1, 11), (0, 1, 12), (2, 1, 15)]:
        with torch.no_grad():
            up, down = x.detach().clone(), x.detach().clone()
            up[at] += h
            down[at] -= h
            d = A.rotary(up, p, t, layout, sections).double() - A.rotary(down, p, t, layout, sections).double()
        slope = float((d * w.double()).sum() / (2 * h))
        # at most two outputs change, each rounded three times from magnitudes below 8
        assert abs(slope - float(x.grad[at])) <= 2 * 2 * 3 * U32 * 8 * float(w.abs().max()) / (2 * h) + 4 * U32 * 8


def test_positions_outside_the_table_are_nan(gpu_lib):
    t = torch.ones(4, 16, 2, device=DEV)
    x = torch.ones(5, 2, 64, device=DEV, dtype=torch.bfloat16)
    p = torch.tensor([0, 3, 4, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y = A.rotary(x, p, t)
    assert torch.isfinite(y[:2]).all() and torch.isnan(y[2:, :, :32]).all()
    assert torch.equal(y[:, :, 32:], x[:, :, 32:])
    two = torch.stack([torch.zeros_like(p), p], 1)
    y = A.rotary(x, two, t, "interleaved", (6, 10))
    assert torch.isfinite(y[:, :, :12]).all() and torch.isnan(y[2:, :, 12:32]).all()


@pytest.mark.parametrize("kw", [dict(), dict(base=1e6), dict(scaling="yarn", factor=32.0, original_len=4096.0)])
def test_table(gpu_lib, kw):
    rot, length = 128, 131072
    f = A.rotary_frequencies(rot, **kw)
    table = A.rotary_table(f, length, DEV).double().cpu().numpy()
    for p in (0, 1, 2, 1000, 65537, length - 1):
        angle = p * f.freq
        # one rounding to float32; the double angle p f is off by 2^-53 p f radians
        bound = (U32 + 2.0 ** -52 * angle + 1e-15) * f.amplitude
        assert (np.abs(table[p, :, 0] - f.amplitude * np.cos(angle)) <= bound).all()
        assert (np.abs(table[p, :, 1] - f.amplitude * np.sin(angle)) <= bound).all()


def test_refusals_and_empty(gpu_lib):
    t = torch.zeros(4, 16, 2, device=DEV)
    p = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.zeros(3, 2, 64, device=DEV)
    assert A.rotary(x[:0], p[:0], t).shape == (0, 2, 64)
    for bad in (dict(x=x.half()), dict(x=x.transpose(1, 2)), dict(x=x[0]), dict(positions=p.long()),
                dict(positions=p[:2]), dict(table=t.double()), dict(table=t[..., :1]), dict(sections=(8, 9)),
                dict(out=x.bfloat16()), dict(x=x[..., :16])):
        with pytest.raises(ValueError):
            A.rotary(**{**dict(x=x, positions=p, table=t), **bad})


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_of_a_gradient(gpu_lib, layout):
    """With y = R x and L = sum(w y^2) / 2 the gradient is g = R' (w y), and the gradient of
    sum(u g) with respect to x is R' (w (R u)): both turns once more, as a gradient penalty
    needs them."""
    rng = np.random.default_rng(16)
    tokens, heads, dim, sections = 5, 3, 32, (4, 8)
    table = _table(rng, 20, 12)
    pos = rng.integers(0, 20, (tokens, 2)).astype(np.int32)
    t, p = torch.from_numpy(table).to(DEV), torch.from_numpy(pos).to(DEV)
    x, w, u = (torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DEV) for _ in range(3))
    x.requires_grad_()
    w.requires_grad_()
    y = A.apply_rotary(x, p, t, layout, sections)
    g, = torch.autograd.grad((w * y * y).sum() / 2, x, create_graph=True)
    gx, gw = torch.autograd.grad((g * u).sum(), (x, w))
    wd, ud, xd = (v.detach().double().cpu().numpy() for v in (w, u, x))
    args = (pos, table, layout, sections)
    ru, mag = AO.rotary(ud, *args)
    e = 3 * U32 * mag                              # of R u: two products and a sum
    z, ez = wd * ru, np.abs(wd) * e + U32 * np.abs(wd * ru) * 1.01
    ref, rmag = AO.rotary(z, *args, backward=True)
    _, spread = AO.rotary(ez, *args, backward=True)
    assert (np.abs(gx.double().cpu().numpy() - ref) <= spread + 3.1 * U32 * rmag).all()
    # with respect to w: y (R u), where the first gradient's own graph has to reach w too
    ry, ymag = AO.rotary(xd, *args)
    bound = np.abs(ry) * e + np.abs(ru) * 3 * U32 * ymag + 2 * U32 * np.abs(ry * ru) + 1e-12
    assert (np.abs(gw.double().cpu().numpy() - ry * ru) <= bound).all()


def test_second_differentiation_twice(gpu_lib):
    """A gradient's graph is kept and used twice, and a third turn goes the first way again."""
    t = torch.from_numpy(_table(np.random.default_rng(2), 9, 16)).to(DEV)
    p = torch.arange(4, dtype=torch.int32, device=DEV)
    x, v = (torch.randn(4, 2, 32, device=DEV, requires_grad=True) for _ in range(2))
    y = A.apply_rotary(x, p, t)
    g, = torch.autograd.grad(y, x, v, create_graph=True)          # R' v
    assert g.requires_grad and torch.equal(g.detach(), A.rotary_backward(v.detach(), p, t))
    w = torch.randn_like(x)
    for _ in range(2):
        gg, = torch.autograd.grad(g, v, w, retain_graph=True)     # R w
        assert torch.equal(gg, A.rotary(w, p, t))


@pytest.mark.parametrize("pairs,length", [(512, 2 ** 23 + 77), (3, 1431655766 + 5)])
def test_table_of_several_launches(gpu_lib, pairs, length):
    """More entries than 2^32 work-items (34 GB), and rows that a launch's limit is no multiple
    of: positions on both sides of every launch's end, and the last ones."""
    f = A.rotary_frequencies(2 * pairs)
    table = A.rotary_table(f, length, DEV)
    assert table.numel() // 2 > 2 ** 32
    step = 2 ** 31 // pairs
    for at in [p for e in range(step, length + step, step) for p in (e - 1, e, e + 1)] + [0, 1, length - 1]:
        if at >= length:
            continue
        row, angle = table[at].double().cpu().numpy(), at * f.freq
        # as in test_table: one rounding to float32, the double angle off by 2^-53 p f radians
        bound = U32 + 2.0 ** -52 * angle + 1e-15
        assert (np.abs(row[:, 0] - np.cos(angle)) <= bound).all() and (np.abs(row[:, 1] - np.sin(angle)) <= bound).all()
    del table
    torch.cuda.empty_cache()


def test_out_that_overlaps_itself_is_refused(gpu_lib):
    t = torch.zeros(4, 16, 2, device=DEV)
    p = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.zeros(3, 2, 64, device=DEV)
    for out in (torch.empty(3, 1, 64, device=DEV).expand(3, 2, 64), torch.empty(1, 2, 64, device=DEV).expand(3, 2, 64)):
        with pytest.raises(ValueError, match="expanded"):
            A.rotary(x, p, t, out=out)
    A.rotary(x[:1].expand(3, 2, 64), p, t, out=torch.empty_like(x))      # of x any stride will do


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_call_of_several_launches(gpu_lib, dtype):
    """More work-items than one launch's grid counts (2^31): on both sides of the boundary, and
    at the end, the result is that of the same tokens in a call of their own (large enough for
    the same number of heads a thread).  One token's values, seen by all (stride 0), at
    changing positions."""
    dim, tokens = 65, 2 ** 25 + 1000              # a turned pair and 63 copied elements: 64 work-items a token
    t = torch.from_numpy(_table(np.random.default_rng(1), 101, 1)).to(DEV)
    x = torch.randn(1, 1, dim, device=DEV).to(dtype).expand(tokens, 1, dim)
    p = (torch.arange(tokens, device=DEV) % 101).to(torch.int32)
    y = A.rotary(x, p, t)
    edge = 2 ** 31 // 64
    for a, b in ((0, 8192), (edge - 8192, edge + 900), (tokens - 8192, tokens)):
        assert torch.equal(y[a:b], A.rotary(x[a:b], p[a:b], t))
    for a in range(0, tokens, 1 << 22):
        assert (y[a:a + (1 << 22), 0, 2:] == x[0, 0, 2:]).all()
        assert (y[a:a + (1 << 22), 0, :2] == y[:101, 0, :2][p[a:a + (1 << 22)].long()]).all()
    del y
    torch.cuda.empty_cache()
