"""What the adapters' sums hold: infinities as the definition has them, bfloat16 results that are
the float32 ones rounded, gradients that are differences to the last bit."""
import pytest
import torch

from test_gpu_adapters import DEV, _gen, _index, _stack

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
# one launch; a wide block of tokens; mixed tokens of several blocks, each width of ranks; several items of one adapter
SIZES = [(1, 256, 264, 8, 3), (40, 256, 264, 16, 3), (50, 2048, 1032, 32, 5), (64, 256, 264, 64, 3), (300, 256, 1032, 8, 2),
         (300, 128, 520, 40, 5), (200, 128, 264, 128, 3), (700, 128, 264, 16, 1)]


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


def _small(shape, g, top=1):
    """Small whole numbers, none zero: products' sums have few bits, so that of their three parts
    of eight bits the later ones are zeros."""
    t = torch.randint(1, top + 1, shape, generator=g, device=DEV)
    return (t * (2 * torch.randint(0, 2, shape, generator=g, device=DEV) - 1)).to(torch.bfloat16)


def _same(got, want):
    """Equal where the definition gives a number, and the same infinity or NaN where it gives one."""
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), (int(got.isnan().sum()), int(want.isnan().sum()))
    assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())


def _products(c, p):
    """c @ p in float64 with every infinity and NaN as one element after another gives it."""
    return (c[:, :, None] * p[None]).sum(1) if c.shape[0] * p.numel() < 2e8 else torch.cat(
        [(row[:, :, None] * p[None]).sum(1) for row in c.split(16)])


@pytest.mark.parametrize("m,k,n,rank,count", SIZES)
@pytest.mark.parametrize("out", TYPES)
def test_infinite_weights(L, m, k, n, rank, count, out):
    g = _gen(m + k)
    x = _small((m, k), g)
    down = _small((count, rank, k), g)
    down[:, :, 2] = 0                                       # k - 1 odd terms: h is never 0
    up = _small((count, rank, n), g, 3)
    up[0, 1, 5], up[0, 2, 6], up[count - 1, 3, n - 1] = float("inf"), -float("inf"), float("nan")
    up[count - 1, 0, 7], up[count - 1, 4, 7] = float("inf"), float("inf")
    a = L.Adapters(down, up, torch.ones(count, device=DEV))
    index = _index("mixed", m, count, g) if m > 1 else torch.zeros(1, dtype=torch.int32, device=DEV)
    y = _small((m, n), g).to(out)
    got = L.lowrank_add(y, x, a, index, out_dtype=out)
    want = y.double()
    for i in range(count):
        at = torch.nonzero(index == i)[:, 0]
        want[at] += _products(x[at].double() @ down[i].double().T, up[i].double())
    assert want.isinf().any()
    _same(got, want)
    fine = want.isfinite()
    assert torch.equal(got[fine].double(), want[fine].to(out).double())       # whole numbers: nothing is rounded before


@pytest.mark.parametrize("m,k,n,rank,count", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_infinite_gradients(L, m, k, n, rank, count, kind):
    g = _gen(m + n)
    x, dy = _small((m, k), g), _small((m, n), g)
    down, up = _small((count, rank, k), g), _small((count, rank, n), g)
    t = m // 2
    dy[t, 3], x[t, 4] = float("inf"), -float("inf")
    down[0, 1, 6] = float("inf")
    a = L.Adapters(down, up, torch.full((count,), 0.5, device=DEV))
    index = _index("mixed", m, count, g) if m > 1 else torch.zeros(1, dtype=torch.int32, device=DEV)
    index[t] = 0
    dx, ddown, dup = L.lowrank_backward(dy, x, a, index, dx_dtype=kind, grad_dtype=kind)
    want = torch.zeros((m, k), dtype=torch.float64, device=DEV)
    for i in range(count):
        at = torch.nonzero(index == i)[:, 0]
        xd, dd, ud, wd = (v.double() for v in (x[at], dy[at], up[i], down[i]))
        h, e = _products(xd, wd.T) * 0.5, _products(dd, ud.T) * 0.5
        want[at] = _products(e, wd)
        _same(ddown[i], _products(e.T, xd))
        _same(dup[i], _products(h.T, dd))
    _same(dx, want)


@pytest.mark.parametrize("m,k,n,rank,count", SIZES)
def test_a_bfloat16_result_is_the_float32_one_rounded(L, m, k, n, rank, count):
    g = _gen(m)
    a = _stack(L, count, rank, k, n, g)
    x = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    index = _index("mixed", m, count, g)
    y = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    for base in (y, y.float()):
        exact = L.lowrank_add(base, x, a, index, out_dtype=torch.float32)
        assert torch.equal(L.lowrank_add(base, x, a, index, out_dtype=torch.bfloat16), exact.to(torch.bfloat16))
    dx = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    exact = L.lowrank_backward(dy, x, a, index, dx=dx.float(), grad_dtype=torch.float32)
    got = L.lowrank_backward(dy, x, a, index, dx=dx, grad_dtype=torch.bfloat16)
    for name, r, e in zip(("dx", "d_down", "d_up"), got, exact):
        assert torch.equal(r, e.to(torch.bfloat16)), (name, int((r != e.to(torch.bfloat16)).sum()), r.numel())


def test_gradients_are_differences_to_the_last_bit(L, gpu_lib):
    """A layer whose weights, adapters, inputs and steps are small whole numbers: every sum is exact in
    float32 and every gradient in bfloat16, and the output is linear in each tensor, so the
    difference of two outputs is the gradient times the step, bit for bit."""
    from w4a16_linear_amd.module import AdaptedLinear, OPQLinear
    k, n, m, rank, count = 96, 64, 40, 8, 3
    g = _gen(21)

    def some(shape, share):                                 # -1, 0 and 1
        return (torch.randint(-1, 2, shape, generator=g, device=DEV) *
                (torch.rand(shape, generator=g, device=DEV) < share)).to(torch.bfloat16)

    lin = torch.nn.Linear(k, n, bias=False).to(DEV)
    with torch.no_grad():
        w = some((n, k), 0.7)
        w[:, 0] = 1                                         # the row's maximum: codes give -1, 0 and 1 back
        lin.weight.copy_(w)
    layer = AdaptedLinear(OPQLinear.from_linear(lin), count, rank)
    assert torch.equal(layer.base.dequantized_weight(), w)
    with torch.no_grad():
        layer.down.copy_(some((count, rank, k), 0.6))
        layer.up.copy_(some((count, rank, n), 0.6))
        layer.scale.copy_(torch.tensor([0.5, 1.0, 2.0]))
    index = _index("mixed", m, count, g)
    assert {0, 1, 2} <= set(index.tolist())
    c = some((m, n), 0.3).float()
    x = some((m, k), 0.8).float().requires_grad_()

    def loss():
        return (layer(x, index).double() * c.double()).sum()

    loss().backward()
    for t, grad in ((layer.down, layer.down.grad), (layer.up, layer.up.grad), (x, x.grad)):
        assert 4 < grad.abs().max() <= 128 and torch.equal(grad * 2, (grad * 2).round())    # halves: exact in bfloat16
        steps = [some(t.shape, 0.5).to(t.dtype) for _ in range(6)]
        for place in torch.randint(0, t.numel(), (20,), generator=g, device=DEV).tolist():  # and element by element
            one = torch.zeros_like(t)
            one.view(-1)[place] = 1
            steps.append(one)
        met = 0
        for step in steps:
            with torch.no_grad():
                t.add_(step)
                up = loss()
                t.sub_(2 * step)
                down = loss()
                t.add_(step)
            want = float((up - down) / 2)
            assert float((grad.double() * step.double()).sum()) == want
            met += want != 0
        assert met >= 16, met                               # a gradient of zeros, or without one term, fails
