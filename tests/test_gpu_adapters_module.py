"""AdaptedLinear and OPQLinear under autograd, streams and graphs on the GPU."""
import copy

import pytest
import torch

from test_gpu_adapters import DEV, HALF, U32, _expected, _gen, _index, _stack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


def _layer(k, n, count, rank, seed=0, **kw):
    from w4a16_linear_amd.module import AdaptedLinear, OPQLinear
    g = _gen(seed)
    lin = torch.nn.Linear(k, n, bias=kw.pop("bias", True)).to(DEV)
    with torch.no_grad():
        lin.weight.copy_(torch.randn((n, k), generator=g, device=DEV) * k ** -0.5)
    layer = AdaptedLinear(OPQLinear.from_linear(lin, **kw), count, rank)
    with torch.no_grad():
        layer.up[:, :rank].copy_(torch.randn((count, rank, n), generator=g, device=DEV) * 0.1)
        layer.scale.copy_(torch.rand(count, generator=g, device=DEV) + 0.5)
    return layer


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", [{}, dict(group_size=32), dict(bits=5), dict(bias=False)])
def test_forward_is_the_base_plus_the_adapters(L, gpu_lib, dtype, form):
    layer = _layer(256, 136, 4, 5, **form)
    x = torch.randn((3, 7, 256), generator=_gen(1), device=DEV).to(dtype)
    with torch.no_grad():
        base = layer.base(x)
        assert torch.equal(layer(x), base)                                     # no index: the base
        index = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
        y = layer(x, index)
        assert torch.equal(y[1], base[1])
        each = index[:, None].expand(3, 7).contiguous()
        assert torch.equal(layer(x, each), y)
        layer.index = index
        assert torch.equal(layer(x), y)
        layer.index = None
    xb = x.reshape(-1, 256).to(torch.bfloat16)
    want, bound = _expected(L, base.reshape(-1, 136), xb, L.Adapters(layer.down.detach(), layer.up.detach(), layer.scale),
                            each.reshape(-1), dtype)
    assert ((y.reshape(-1, 136).double() - want).abs() <= bound).all()
    tracked = layer(x, index)                                                  # parameters require grad: the same numbers
    assert tracked.requires_grad and torch.equal(tracked, y)


@pytest.mark.parametrize("m,k,n,count,rank", [(1, 64, 64, 1, 8), (9, 256, 136, 3, 5), (70, 128, 264, 2, 16), (300, 512, 96, 5, 24)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_are_the_formulas(L, gpu_lib, m, k, n, count, rank, dtype):
    layer = _layer(k, n, count, rank, seed=m)
    g = _gen(m + 1)
    x = torch.randn((m, k), generator=g, device=DEV).to(dtype).requires_grad_()
    index = _index("mixed", m, count, g)
    dy = torch.randn((m, n), generator=g, device=DEV).to(dtype)
    layer(x, index).backward(dy)
    # the formulas in float64, from the tensors as the kernels read them (x and dy in bfloat16)
    xb, db = x.detach().to(torch.bfloat16).double(), dy.to(torch.bfloat16).double()
    w = layer.base.dequantized_weight().double()
    dx, ddown, dup = db @ w, torch.zeros_like(layer.down, dtype=torch.float64), torch.zeros_like(layer.up, dtype=torch.float64)
    slack = (n + 64) * U32 * (db.abs() @ w.abs())
    for i in range(count):
        at = torch.nonzero(index == i)[:, 0]
        s, d, u = layer.scale[i].double(), layer.down[i].detach().double(), layer.up[i].detach().double()
        h, e = s * xb[at] @ d.T, s * db[at] @ u.T
        ddown[i], dup[i] = e.T @ xb[at], h.T @ db[at]
        dx[at] += e @ d
        slack[at] += (n + 2.0 ** 9 + 200) * U32 * ((s * db[at].abs() @ u.abs().T) @ d.abs())  # e's sums, its two bf16 parts
    # each gradient is rounded to its type once; dx is that of the projection first (one more rounding)
    half = 2 * HALF[dtype]
    assert x.grad.dtype == dtype
    assert ((x.grad.double() - dx).abs() <= slack + half * (dx.abs() + slack) + half * (db @ w).abs()).all()
    for got, want, a, b, size in ((layer.down.grad, ddown, db, layer.up, n), (layer.up.grad, dup, xb, layer.down, k)):
        other = xb if a is db else db
        for i in range(count):
            at = torch.nonzero(index == i)[:, 0]
            big = layer.scale[i].double() * (a[at].abs() @ b[i].detach().double().abs().T).T @ other[at].abs()
            off = (size + 2.0 ** 9 + 3 * m + 200) * U32 * big
            assert ((got[i].double() - want[i]).abs() <= off + 2.0 ** -8 * (want[i].abs() + off)).all()
    assert not layer.down.grad[:, rank:].any() and not layer.up.grad[:, rank:].any()     # the padding stays zeros


def test_gradients_are_the_differences(L, gpu_lib):
    """sum(c * y) is linear in up, in down and in x alone, so a step of any size gives the gradient;
    every step here is exact in bfloat16."""
    k, n, m, rank = 128, 64, 40, 8
    layer = _layer(k, n, 2, rank, seed=3)
    g = _gen(9)

    def exact(*shape):                                                          # multiples of 1/8 up to 4, sums exact
        return torch.randint(-16, 17, shape, generator=g, device=DEV).to(torch.bfloat16) / 8

    with torch.no_grad():
        layer.down.copy_(exact(2, rank, k))
        layer.up.copy_(exact(2, rank, n))
        layer.scale.fill_(0.5)
    index = _index("runs", m, 2, g)
    c = exact(m, n).float()
    x = exact(m, k).float().requires_grad_()
    (layer(x, index) * c).sum().backward()
    for t, grad in ((layer.down, layer.down.grad), (layer.up, layer.up.grad), (x, x.grad)):
        step = torch.randint(-8, 9, t.shape, generator=g, device=DEV).to(t.dtype) / 8
        with torch.no_grad():
            t.add_(step)
            up = (layer(x, index).double() * c.double()).sum()
            t.sub_(2 * step)
            down = (layer(x, index).double() * c.double()).sum()
            t.add_(step)
        # A step makes |x|, |down| and |up| at most 3, |c| is at most 2 and the scale 1/2: the terms of an
        # element of y add up to 27/2 k rank and 3 |w|'s row sum at most.  y is a float32 sum of k, rank and
        # two terms, so each side is off by (k + rank + 128) half steps of that; the gradient by half a step
        # of its type, each element (twice for x: the projection's part is rounded first).
        terms = m * n * 2.0 * (13.5 * k * rank + 3.0 * layer.base.dequantized_weight().double().abs().sum(1).max())
        half = 2.0 ** -8 if t is not x else 2 * U32
        got, want = (grad.double() * step.double()).sum(), (up - down) / 2
        bound = 2 * (k + rank + 128) * U32 * terms + half * (grad.double().abs() * step.double().abs()).sum()
        assert abs(got - want) <= bound, (float(got), float(want), float(bound))


def test_linear_passes_gradients_through(L, gpu_lib):
    from w4a16_linear_amd.module import OPQLinear
    lin = torch.nn.Linear(256, 100).to(DEV)
    for form in ({}, dict(group_size=64), dict(bits=3)):
        layer = OPQLinear.from_linear(lin, **form)
        x = torch.randn((2, 5, 256), generator=_gen(2), device=DEV).requires_grad_()
        y = layer(x)
        with torch.no_grad():
            assert torch.equal(layer(x), y) and not layer(x).requires_grad
        dy = torch.randn(y.shape, generator=_gen(3), device=DEV)
        y.backward(dy)
        w = layer.dequantized_weight().double()
        db = dy.to(torch.bfloat16).double()
        want, bound = db @ w, (100 + 64) * U32 * (db.abs() @ w.abs())
        assert ((x.grad.double() - want).abs() <= bound + U32 * want.abs()).all()


def test_what_autograd_refuses(L, gpu_lib):
    layer = _layer(64, 64, 2, 8)
    x = torch.randn((3, 64), device=DEV, requires_grad=True)
    index = torch.zeros(3, dtype=torch.int32, device=DEV)
    y = layer(x, index)
    (gx,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()                                                     # gradients of gradients
    stack = layer.stack()
    xb = x.detach().to(torch.bfloat16)
    with pytest.raises(RuntimeError, match="requires grad"):
        L.lowrank_add(None, xb, stack, index)
    with pytest.raises(RuntimeError, match="requires grad"):
        L.linear_backward(xb.clone().requires_grad_(), layer.base.qweight(), 0.73)
    with pytest.raises(RuntimeError, match="scale"):
        L.apply_adapted(x, layer.base.qweight(), 0.73, None, stack._replace(scale=layer.scale.clone().requires_grad_()), index)
    z = layer(x, index)
    layer.base.mx.mul_(1)                                                       # the weights changed under a graph
    with pytest.raises(RuntimeError, match="modified"):
        z.sum().backward()
    frozen = _layer(64, 64, 2, 8)
    frozen.down.requires_grad_(False)
    frozen.up.requires_grad_(False)
    out = frozen(x, index)
    out.sum().backward()                                                        # only x's gradient
    assert frozen.down.grad is None and x.grad is not None


def test_written_memory_is_known(L):
    a = _stack(L, 2, 8, 64, 32, _gen(0))
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    index = torch.zeros(4, dtype=torch.int32, device=DEV)
    y = torch.zeros((4, 32), device=DEV)
    before = y._version
    assert L.lowrank_add(y, x, a, index, out=y) is y and y._version > before
    dx = torch.zeros((4, 64), device=DEV)
    before = dx._version
    got, _, _ = L.lowrank_backward(y.bfloat16(), x, a, index, dx=dx, out=dx)
    assert got is dx and dx._version > before


def test_strides_and_shared_memory(L):
    g = _gen(4)
    a = _stack(L, 3, 16, 96, 64, g)
    index = _index("mixed", 50, 3, g)
    wide = torch.randn((50, 320), generator=g, device=DEV).to(torch.bfloat16)
    x, y = wide[:, 8:104], wide[:, 128:192]
    want = L.lowrank_add(y.contiguous(), x.contiguous(), a, index)
    assert torch.equal(L.lowrank_add(y, x, a, index), want)
    kept = wide.clone()
    out = wide[:, 200:264]
    assert torch.equal(L.lowrank_add(y, x, a, index, out=out), want)            # beside its inputs
    kept[:, 200:264] = want
    assert torch.equal(wide, kept)
    assert torch.equal(L.lowrank_add(y, x, a, index, out=y), want)              # in place, the rest untouched
    kept[:, 128:192] = want
    assert torch.equal(wide, kept)
    same = x[:1].expand(50, 96)                                                 # one row for all tokens
    assert torch.equal(L.lowrank_add(None, same, a, index), L.lowrank_add(None, same.contiguous(), a, index))
    for bad in (lambda: L.lowrank_add(y, x, a, index, out=wide[:, 132:196]), lambda: L.lowrank_add(y, x, a, index, out=wide[:, 96:160]),
                lambda: L.lowrank_add(y, x, a, index, out=wide[1:2, 200:264].expand(50, 64)),
                lambda: L.lowrank_add(y, x.t(), a, index), lambda: L.lowrank_add(y, x, a, index[:49].contiguous()),
                lambda: L.lowrank_add(y, x, a, index.long()), lambda: L.lowrank_add(y[:, :56], x, a, index),
                lambda: L.lowrank_add(wide[:, 3:67], x, a, index), lambda: L.lowrank_add(y, x.float(), a, index),
                lambda: L.lowrank_add(y, x, a._replace(down=a.down.float()), index), lambda: L.lowrank_add(y, x, a[:2], index),
                lambda: L.lowrank_add(y, x, a, index, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
                lambda: L.lowrank_add(y, x, a, index, out=torch.empty((50, 64), dtype=torch.float16, device=DEV)),
                lambda: L.lowrank_backward(y, x, a, index, dx=x, out=wide[:, 16:112])):
        with pytest.raises(ValueError):
            bad()


def test_values_that_spread(L):
    """Infinities and NaN stay with their tokens; huge and tiny values survive the split in parts."""
    g = _gen(6)
    m, k, n = 70, 64, 48
    a = _stack(L, 3, 8, k, n, g)
    x = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    y = torch.randn((m, n), generator=g, device=DEV)
    index = _index("mixed", m, 3, g)
    clean = L.lowrank_add(y, x, a, index)
    hurt = x.clone()
    hurt[5], hurt[17, 3], hurt[33] = float("nan"), float("inf"), -float("inf")
    got = L.lowrank_add(y, hurt, a, index)
    rest = torch.ones(m, dtype=torch.bool, device=DEV)
    rest[[5, 17, 33]] = False
    assert torch.equal(got[rest], clean[rest])
    for t in (5, 17, 33):
        i = int(index[t])
        if i < 0:
            assert torch.equal(got[t], y[t])
        else:
            assert not torch.isfinite(got[t]).any()
    none = torch.full_like(index, -1)
    assert torch.equal(L.lowrank_add(y, hurt, a, none), y)                      # no adapter: x is not looked at
    bad = a._replace(down=a.down.clone())
    bad.down[2] = float("nan")                                                  # an adapter no token uses
    two = torch.where(index == 2, 1, index)
    assert torch.equal(L.lowrank_add(y, x, bad, two), L.lowrank_add(y, x, a, two))
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    _, down, up = L.lowrank_backward(dy, x, bad, two)
    _, down0, up0 = L.lowrank_backward(dy, x, a, two)
    assert torch.equal(down, down0) and torch.equal(up, up0)
    for scale in (2.0 ** 100, 2.0 ** -100):
        one = torch.zeros_like(index)
        big = L.lowrank_add(None, (x.float() * scale).to(torch.bfloat16), a, one, out_dtype=torch.float32)
        assert torch.equal(big, L.lowrank_add(None, x, a, one, out_dtype=torch.float32) * scale)


def test_streams(L):
    """Calls on two streams at once, each with inputs made there, give what one stream gives."""
    g = _gen(8)
    a = _stack(L, 4, 16, 512, 1024, g)
    sets = []
    for m in (33, 700):
        x = torch.randn((m, 512), generator=g, device=DEV).to(torch.bfloat16)
        sets.append((x, torch.randn((m, 1024), generator=g, device=DEV).to(torch.bfloat16), _index("mixed", m, 4, g)))
    want = [(L.lowrank_add(y, x, a, i), L.lowrank_backward(y, x, a, i)) for x, y, i in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                x, y, i = (t.clone() for t in sets[s])
                got[s].append((L.lowrank_add(y, x, a, i), L.lowrank_backward(y, x, a, i)))
    torch.cuda.synchronize()
    for s in range(2):
        for add, back in got[s]:
            assert torch.equal(add, want[s][0])
            assert all(torch.equal(b, w) for b, w in zip(back, want[s][1]))


@pytest.mark.parametrize("m", [5, 300])
def test_in_a_graph(L, gpu_lib, m):
    """Add, backward and the projection's gradient captured: replays on new contents equal eager calls."""
    layer = _layer(256, 128, 4, 16, seed=m)
    a = L.Adapters(layer.down.detach(), layer.up.detach(), layer.scale)
    w = layer.base.qweight()
    g = _gen(m)

    def new():
        return (torch.randn((m, 256), generator=g, device=DEV).to(torch.bfloat16),
                torch.randn((m, 128), generator=g, device=DEV).to(torch.bfloat16), _index("mixed", m, 4, g))

    def step(x, y, i):
        out = L.lowrank_add(y, x, a, i)
        dx = L.linear_backward(out, w, 0.73)
        return (out, *L.lowrank_backward(out, x, a, i, dx=dx, out=dx))

    x, y, i = new()
    step(x, y, i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(x, y, i)
    for _ in range(4):
        for t, v in zip((x, y, i), new()):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = step(x, y, i)
        torch.cuda.synchronize()
        assert all(torch.equal(r, e) for r, e in zip(res, want))


@pytest.mark.parametrize("n", [10, 1000])
def test_gradients_that_start_anywhere(gpu_lib, n):
    """What a backward pass hands on may be a part of a longer tensor: of a concatenation's, say."""
    from w4a16_linear_amd.module import AdaptedLinear, OPQLinear
    lin = torch.nn.Linear(64, n).to(DEV)
    base = OPQLinear.from_linear(lin)
    g = _gen(n)
    x = torch.randn((7, 64), generator=g, device=DEV).to(torch.bfloat16).requires_grad_()
    dy = torch.randn((7, n), generator=g, device=DEV).to(torch.bfloat16)
    layers = [base] if n % 8 else [base, AdaptedLinear(base, 2, 8)]
    for layer in layers:
        args = () if layer is base else (torch.zeros(7, dtype=torch.int32, device=DEV),)
        (want,) = torch.autograd.grad(layer(x, *args), x, dy)
        long = torch.empty(7 * n + 3, dtype=torch.bfloat16, device=DEV)
        for start in (1, 3):
            odd = long[start:start + 7 * n].view(7, n)
            odd.copy_(dy)
            (got,) = torch.autograd.grad(layer(x, *args), x, odd)
            assert torch.equal(got, want)
        (got,) = torch.autograd.grad(torch.cat((layer(x[:3], *(a[:3] for a in args)), layer(x[3:], *(a[3:] for a in args)))), x, dy)
        (a,) = torch.autograd.grad(layer(x[:3], *(a[:3] for a in args)), x, dy[:3].clone())
        (b,) = torch.autograd.grad(layer(x[3:], *(a[3:] for a in args)), x, dy[3:].clone())
        assert torch.equal(got, a + b)


def test_layers_made_in_inference_mode(gpu_lib):
    """Codes made under inference_mode have no versions to watch; gradients pass through them all the same."""
    from w4a16_linear_amd.module import AdaptedLinear, OPQLinear
    lin = torch.nn.Linear(64, 32).to(DEV)
    with torch.inference_mode():
        base = OPQLinear.from_linear(lin)
    plain = OPQLinear.from_linear(lin)
    x = torch.randn((5, 64), device=DEV, requires_grad=True)
    (want,) = torch.autograd.grad(plain(x).sum(), x)
    (got,) = torch.autograd.grad(base(x).sum(), x)
    assert torch.equal(got, want)
    layer = AdaptedLinear(base, 2, 8)
    with torch.no_grad():
        layer.up.normal_()
    layer(x, torch.zeros(5, dtype=torch.int32, device=DEV)).sum().backward()
    assert layer.down.grad.isfinite().all() and layer.down.grad.any() and x.grad is not None


def test_layers_share_no_workspace(L, gpu_lib, monkeypatch):
    """Layers of one model on two streams at once: every forward has a workspace of its own."""
    from w4a16_linear_amd.module import OPQLinear
    m = 700                                                                     # a split contraction, or W' decoded beside
    sets = []
    for s, form in enumerate(({}, dict(bits=5))):
        layer = _layer(2048, 256, 3, 8, seed=s, **form)
        x = torch.randn((m, 2048), generator=_gen(s), device=DEV).to(torch.bfloat16)
        index = _index("mixed", m, 3, _gen(s))
        y = gpu_lib.linear(x, layer.base.qweight(), layer.base.alpha, bias=layer.base.bias, out_dtype=torch.bfloat16)
        with torch.no_grad():
            sets.append((layer, x, index, y, L.lowrank_add(y, x, layer.stack(), index)))
    assert all(gpu_lib.linear_workspace_bytes(m, 256, 2048, bits) for bits in (4, 5))
    monkeypatch.setattr(gpu_lib, "shared_workspace", lambda *a: pytest.fail("a workspace that others use"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for s, stream in enumerate(streams):
            layer, x, index, _, _ = sets[s]
            with torch.cuda.stream(stream):
                tracked = x.detach().clone().requires_grad_()
                with torch.no_grad():
                    got[s].append((layer.base(x), layer(x, index)))
                got[s].append((layer.base(tracked).detach(), layer(tracked, index).detach()))
    torch.cuda.synchronize()
    for s in range(2):
        for base, adapted in got[s]:
            assert torch.equal(base, sets[s][3]) and torch.equal(adapted, sets[s][4])


@pytest.mark.parametrize("m", [6, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_training_step_in_a_graph(L, gpu_lib, m, dtype):
    """Two adapted layers, forward, backward and update captured together: replays on new inputs, with
    eager work between, leave the parameters that eager steps leave."""
    layers = [_layer(128, 256, 3, 8, seed=1, bits=5), _layer(256, 64, 3, 5, seed=2)]
    eager, fresh = copy.deepcopy(layers), copy.deepcopy(layers)
    x, dy = (torch.zeros((m, w), dtype=dtype, device=DEV) for w in (128, 64))
    index = torch.zeros(m, dtype=torch.int32, device=DEV)

    def step(layers):
        h = torch.relu(layers[0](x, index))
        layers[1](h, index).backward(dy)
        with torch.no_grad():
            for layer in layers:
                for p in (layer.down, layer.up):
                    p.sub_(0.01 * p.grad)
        for layer in layers:
            layer.down.grad = layer.up.grad = None

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(layers)                                                        # of zeros: the parameters stay
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layers)
    g = _gen(m)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        dy.copy_(torch.randn(dy.shape, generator=g, device=DEV))
        index.copy_(_index("mixed", m, 3, g))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for a, b in zip(layers, eager):
            assert torch.equal(a.down, b.down) and torch.equal(a.up, b.up)
    assert not torch.equal(layers[0].down, fresh[0].down) and not torch.equal(layers[1].up, fresh[1].up)
