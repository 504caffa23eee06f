"""Low-rank adapters and their gradients on the GPU against float64, within bounds that
follow from the roundings include/opq_adapters.h states."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
U32 = 2.0 ** -24                     # half a step of float32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
# what two bfloat16 parts leave of a float32: the first, cut off, leaves less than 2^-7 of it,
# of which the second, rounded, leaves 2^-8; three parts hold all 24 bits
LEFT = {torch.bfloat16: 2.0 ** -15, torch.float32: 0.0}


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _index(kind, m, count, g):
    if kind == "one":
        i = torch.zeros(m, dtype=torch.long, device=DEV) + min(1, count - 1)
    elif kind == "runs":
        i = (torch.arange(m, device=DEV) * min(count, 3)) // max(1, m)
    elif kind == "mixed":
        i = torch.randint(-1, count, (m,), generator=g, device=DEV)
    elif kind == "outside":
        i = torch.randint(-2, count + 2, (m,), generator=g, device=DEV)
        i = torch.where(i >= count, i + 2 ** 30, i)
    else:
        i = torch.full((m,), -1, device=DEV)
    return i.to(torch.int32)


def _stack(L, count, rank, k, n, g):
    down = (torch.randn((count, rank, k), generator=g, device=DEV) * k ** -0.5).to(torch.bfloat16)
    up = torch.randn((count, rank, n), generator=g, device=DEV).to(torch.bfloat16) * 0.25
    return L.Adapters(down, up, torch.rand(count, generator=g, device=DEV) + 0.5)


def _shrink(v, p, d):
    """(c, bound): c_t = P v_t in float64, and how far sums of d products in float32 may be off
    (every partial sum is at most the sum of magnitudes, and there are fewer than d + 64 of them)."""
    c = v.double() @ p.double().T
    return c, (d + 64) * U32 * (v.double().abs() @ p.double().abs().T)


def _expected(L, y, x, a, index, out):
    """(result, bound) of lowrank_add in float64."""
    k, rank = a.down.shape[2], a.down.shape[1]
    r = torch.zeros((x.shape[0], a.up.shape[2]), dtype=torch.float64, device=DEV) if y is None else y.double()
    bound = torch.zeros_like(r)
    for i in range(a.down.shape[0]):
        at = torch.nonzero(index == i)[:, 0]
        if at.numel() == 0:
            continue
        s, up = a.scale[i].double(), a.up[i].double()
        h, dh = _shrink(x[at], a.down[i], k)
        h, dh = s * h, s * (dh + 2 * U32 * h.abs())              # the product with s, the slices' sum
        r[at] += h @ up
        size = (h.abs() + dh) @ up.abs()
        bound[at] += dh @ up.abs() + (LEFT[out] + (3 * rank + 16) * U32) * size
        bound[at] += U32 * (r[at].abs() + size)                  # the sum with y
    return r, bound + HALF[out] * (r.abs() + bound)


CASES = [  # m, k, n, rank, adapters, index
    (1, 3840, 3840, 8, 4, "one"), (1, 8, 8, 8, 1, "one"), (2, 40, 136, 16, 3, "mixed"), (17, 256, 520, 24, 5, "mixed"),
    (48, 3840, 1152, 16, 64, "mixed"), (33, 1000, 1000, 32, 2, "runs"), (64, 512, 96, 64, 7, "outside"),
    (256, 736, 640, 40, 300, "mixed"), (257, 288, 264, 128, 3, "runs"), (130, 96, 2048, 128, 9, "mixed"),
    (777, 1056, 904, 72, 4, "runs"), (1025, 320, 384, 16, 1, "one"), (600, 64, 512, 8, 2, "none"),
    (515, 2048, 128, 48, 40, "outside"),
    # one launch for few tokens, and past each of its limits
    (50, 2048, 2056, 32, 6, "mixed"), (64, 72, 4104, 8, 70, "outside"), (48, 2056, 264, 32, 5, "mixed"),
    (64, 64, 8456, 16, 9, "outside"), (65, 136, 72, 24, 4, "one"),
]


@pytest.mark.parametrize("m,k,n,rank,count,kind", CASES)
@pytest.mark.parametrize("y_type,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                        (None, torch.bfloat16), (torch.bfloat16, torch.float32),
                                        (torch.float32, torch.bfloat16)])
def test_add(L, m, k, n, rank, count, kind, y_type, out):
    g = _gen(m * 7 + k + rank)
    a = _stack(L, count, rank, k, n, g)
    x = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    y = None if y_type is None else torch.randn((m, n), generator=g, device=DEV).to(y_type)
    index = _index(kind, m, count, g)
    got = L.lowrank_add(y, x, a, index, out_dtype=out)
    want, bound = _expected(L, y, x, a, index, out)
    assert got.dtype == out and got.shape == (m, n)
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() - bound).max())
    alone = (index < 0) | (index >= count)                      # y as it was, converted
    if y is not None:
        assert torch.equal(got[alone], y[alone].to(out))
    else:
        assert not got[alone].any()
    again = L.lowrank_add(y, x, a, index, out_dtype=out)
    assert torch.equal(got, again)


GRADS = [c for c in CASES if c[0] > 1 and c[4] <= 64]


@pytest.mark.parametrize("m,k,n,rank,count,kind", GRADS + [(4096, 256, 264, 16, 2, "runs"), (1, 64, 64, 8, 3, "one")])
@pytest.mark.parametrize("dx_type,grad", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_backward(L, m, k, n, rank, count, kind, dx_type, grad):
    g = _gen(m * 5 + n + rank)
    a = _stack(L, count, rank, k, n, g)
    x = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    dx0 = torch.randn((m, k), generator=g, device=DEV).to(dx_type)
    index = _index(kind, m, count, g)
    dx, down, up = L.lowrank_backward(dy, x, a, index, dx=dx0, grad_dtype=grad)
    want, bound = dx0.double(), torch.zeros((m, k), dtype=torch.float64, device=DEV)
    for i in range(count):
        at = torch.nonzero(index == i)[:, 0]
        if at.numel() == 0:
            assert not down[i].any() and not up[i].any()
            continue
        s, t = a.scale[i].double(), at.numel()
        h, dh = _shrink(x[at], a.down[i], k)
        e, de = _shrink(dy[at], a.up[i], n)
        h, dh = s * h, s * (dh + 4 * U32 * h.abs())
        e, de = s * e, s * (de + 4 * U32 * e.abs())
        p = a.down[i].double()
        want[at] += e @ p
        size = (e.abs() + de) @ p.abs()
        bound[at] += de @ p.abs() + (LEFT[dx_type] + (3 * rank + 16) * U32) * size + U32 * (want[at].abs() + size)
        for got, c, dc, v in ((down[i], e, de, x[at].double()), (up[i], h, dh, dy[at].double())):
            exact = c.T @ v
            big = (c.abs() + dc).T @ v.abs()
            off = dc.T @ v.abs() + (LEFT[grad] + (3 * t + 64) * U32) * big
            off = off + HALF[grad] * (exact.abs() + off)
            assert ((got.double() - exact).abs() <= off).all(), (i, float(((got.double() - exact).abs() - off).max()))
    bound = bound + HALF[dx_type] * (want.abs() + bound)
    assert ((dx.double() - want).abs() <= bound).all(), float(((dx.double() - want).abs() - bound).max())
    only, none1, none2 = L.lowrank_backward(dy, x, a, index, dx=dx0, adapter_grads=False)
    assert torch.equal(only, dx) and none1 is None and none2 is None
    nodx, down2, up2 = L.lowrank_backward(dy, x, a, index, input_grad=False, grad_dtype=grad)
    assert nodx is None and torch.equal(down2, down) and torch.equal(up2, up)


def test_no_tokens(L):
    a = _stack(L, 3, 16, 64, 32, _gen(0))
    x, dy = (torch.empty((0, w), dtype=torch.bfloat16, device=DEV) for w in (64, 32))
    index = torch.empty(0, dtype=torch.int32, device=DEV)
    assert L.lowrank_add(dy, x, a, index).shape == (0, 32)
    dx, down, up = L.lowrank_backward(dy, x, a, index)
    assert dx.shape == (0, 64) and not down.any() and not up.any()
    none = L.Adapters(a.down[:0], a.up[:0], a.scale[:0])
    y = torch.randn((5, 32), device=DEV)
    at = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert torch.equal(L.lowrank_add(y, torch.ones((5, 64), dtype=torch.bfloat16, device=DEV), none, at), y)


# Long rows in few slices, so that a wave takes whole runs of steps, and tiles of every width: up to 16
# tokens of an adapter, up to 32 and up to 64, each size of ranks, a block of tokens alone and many
LONG = [(m, 2088, n, rank, count) for m, n in ((16400, 40), (64, 10248)) for rank in (8, 16, 24, 64, 128)
        for count in ((5, 2, 1) if m > 64 else (60, 3, 1))]


@pytest.mark.parametrize("m,k,n,rank,count", LONG)
def test_long_rows(L, m, k, n, rank, count):
    test_add(L, m, k, n, rank, count, "mixed", torch.bfloat16, torch.float32)
    test_add(L, m, n, k, rank, count, "mixed", None, torch.float32)


@pytest.mark.parametrize("m,k,n,rank,count", LONG + [(4096, 32, 11520, 16, 3), (2049, 4096, 4104, 8, 3), (20000, 24, 4096, 8, 3)])
def test_gradients_of_long_rows(L, m, k, n, rank, count):
    test_backward(L, m, k, n, rank, count, "mixed", torch.float32, torch.float32)
    test_backward(L, m, n, k, rank, count, "mixed", torch.bfloat16, torch.bfloat16)
