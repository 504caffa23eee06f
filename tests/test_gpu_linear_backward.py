"""The gradient through a quantized projection on the GPU against float64 products with the
very weights opq_dequantize writes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


def _weight(opq, n, k, form, alpha, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + n + k)
    w = torch.randn((n, k), generator=g, device=DEV) * 0.02
    if form == "row":
        return opq.quantize(w, alpha)
    if isinstance(form, str):
        return opq.quantize_bits(w, alpha, int(form[0]))
    return opq.quantize_grouped(w, alpha, form)


@pytest.mark.parametrize("m,n,k", [(1, 32, 32), (7, 1, 32), (33, 100, 256), (64, 31, 512), (65, 264, 256), (130, 1000, 768),
                                   (257, 96, 512), (300, 520, 1024), (333, 3840, 512), (1024, 200, 256),
                                   (5, 264, 96), (64, 1000, 160), (17, 7, 224), (16, 2000, 1280), (40, 777, 640), (3, 5000, 128),
                                   (140, 5, 96), (256, 1023, 160), (385, 96, 32), (512, 300, 544)])
@pytest.mark.parametrize("form", ["row", 32, 128, "3b", "5b"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear_backward(L, gpu_lib, m, n, k, form, out):
    opq, alpha = gpu_lib, 0.73
    if isinstance(form, int) and k % form:
        pytest.skip("groups do not tile k")
    w = _weight(opq, n, k, form, alpha)
    g = torch.Generator(device=DEV)
    g.manual_seed(m + n + k)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    got = L.linear_backward(dy, w, alpha, out_dtype=out)
    full = opq.dequantize(w, alpha).double()
    want = dy.double() @ full
    # sums of n products in float32, one rounding to the result's type
    bound = (n + 64) * 2.0 ** -24 * (dy.double().abs() @ full.abs())
    bound = bound + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24) * (want.abs() + bound)
    assert got.dtype == out and got.shape == (m, k)
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() - bound).max())
    assert torch.equal(got, L.linear_backward(dy, w, alpha, out_dtype=out))


@pytest.mark.parametrize("m", [31, 100, 128, 129, 256, 257, 384, 385, 512, 513])
@pytest.mark.parametrize("form", ["row", 64, 256])
def test_at_the_change_of_paths(L, gpu_lib, m, form):
    opq, alpha, n, k = gpu_lib, 0.73, 1100, 768
    w = _weight(opq, n, k, form, alpha)
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    got = L.linear_backward(dy, w, alpha, out_dtype=torch.float32).double()
    full = opq.dequantize(w, alpha).double()
    want = dy.double() @ full
    bound = (n + 64) * 2.0 ** -24 * (dy.double().abs() @ full.abs())
    assert ((got - want).abs() <= bound + 2.0 ** -24 * (want.abs() + bound)).all()


@pytest.mark.parametrize("m", [4, 200])
def test_an_infinite_last_row(L, gpu_lib, m):
    """Rows past the last one are not the last one again: an infinity in it stays an infinity."""
    opq, n, k = gpu_lib, 45, 128
    w = _weight(opq, n, k, "row", 1.0)
    w = w._replace(scale=w.scale.clone())
    w.scale[-1] = float("inf")
    full = opq.dequantize(w, 1.0).double()
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    want = dy.double() @ full
    got = L.linear_backward(dy, w, 1.0, out_dtype=torch.float32).double()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isposinf(), want.isposinf())
    assert torch.equal(got.isneginf(), want.isneginf())


@pytest.mark.parametrize("m", [8, 200])
def test_out_beside_dy_not_over_it(L, gpu_lib, m):
    w = _weight(gpu_lib, 256, 256, "row", 0.73)
    held = torch.randn((2 * m, 256), device=DEV).to(torch.bfloat16)
    want = L.linear_backward(held[:m].clone(), w, 0.73)
    assert torch.equal(L.linear_backward(held[:m], w, 0.73, out=held[m:]), want)
    assert torch.equal(held[m:], want)
    for out in (held[:m], held[1:m + 1]):
        with pytest.raises(ValueError, match="share"):
            L.linear_backward(held[:m], w, 0.73, out=out)


def test_every_path_in_a_graph_and_on_a_stream(L, gpu_lib):
    """Captured, replayed on new contents between eager calls, and beside calls on another stream."""
    opq, n, k = gpu_lib, 1100, 768
    w = _weight(opq, n, k, "row", 0.73)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    sizes = (8, 64, 100, 300, 512, 600)
    dys = [torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16) for m in sizes]
    outs = [torch.empty((m, k), dtype=torch.bfloat16, device=DEV) for m in sizes]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for dy, out in zip(dys, outs):
            L.linear_backward(dy, w, 0.73, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for dy, out in zip(dys, outs):
            L.linear_backward(dy, w, 0.73, out=out)
    for _ in range(3):
        for dy in dys:
            dy.copy_(torch.randn(dy.shape, generator=g, device=DEV))
        want = [L.linear_backward(dy, w, 0.73) for dy in dys]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            beside = [L.linear_backward(dy, w, 0.73) for dy in dys]
        graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b, c in zip(want, beside, outs):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("m", [3, 100, 600])
@pytest.mark.parametrize("form", ["row", 128, "5b"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_a_vocabulary_of_rows(L, gpu_lib, m, form, out):
    """More rows than one call of the library takes, as the head of a large vocabulary has."""
    opq, alpha, n, k = gpu_lib, 0.73, 2 * 65536 + 1000, 256
    w = _weight(opq, n, k, form, alpha)
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    dy = torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16)
    got = L.linear_backward(dy, w, alpha, out_dtype=out)
    full = opq.dequantize(w, alpha).double()
    want = dy.double() @ full
    bound = (n + 64) * 2.0 ** -24 * (dy.double().abs() @ full.abs())
    bound = bound + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24) * (want.abs() + bound)
    assert got.dtype == out and ((got.double() - want).abs() <= bound).all()
    # exact sums: every row counts once, and rows of blocks are not mixed up
    one = torch.zeros((m, n), dtype=torch.bfloat16, device=DEV)
    at = torch.randint(0, n, (m,), generator=g, device=DEV)
    one[torch.arange(m, device=DEV), at] = 2.0
    held = torch.empty((m, k), dtype=out, device=DEV)
    room = torch.empty(L.linear_backward_workspace_bytes(m, n, k), dtype=torch.uint8, device=DEV)
    assert L.linear_backward(one, w, alpha, out=held, workspace=room) is held
    assert torch.equal(held.double(), 2.0 * full[at])
    if room.numel():
        with pytest.raises(ValueError):
            L.linear_backward(one, w, alpha, workspace=room[:1])


def test_more_tokens_than_one_call(L, gpu_lib):
    w = _weight(gpu_lib, 8, 32, "row", 0.73)
    m = (1 << 22) + 77
    dy = torch.zeros((m, 8), dtype=torch.bfloat16, device=DEV)
    at = torch.arange(0, m, 4099, device=DEV)
    at = torch.cat((at, torch.tensor([m - 1, m - 77, m - 78], device=DEV)))
    dy[at, at % 8] = 2.0
    got = L.linear_backward(dy, w, 0.73)
    want = torch.zeros((m, 32), dtype=torch.bfloat16, device=DEV)
    want[at] = (2.0 * gpu_lib.dequantize(w, 0.73).double()[at % 8]).to(torch.bfloat16)
    assert torch.equal(got, want)


def test_a_layer_with_a_vocabulary(L, gpu_lib):
    from w4a16_linear_amd.module import AdaptedLinear, OPQLinear
    layer = OPQLinear.from_linear(torch.nn.Linear(64, 70000, bias=False).to(DEV))
    x = torch.randn((5, 64), device=DEV, requires_grad=True)
    dy = torch.randn((5, 70000), device=DEV)
    want = dy.to(torch.bfloat16).double() @ layer.dequantized_weight().double()
    bound = (70000 + 64) * 2.0 ** -24 * (dy.to(torch.bfloat16).double().abs() @ layer.dequantized_weight().double().abs())
    (got,) = torch.autograd.grad(layer(x), x, dy)
    assert ((got.double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
    adapted = AdaptedLinear(layer, 2, 8)                    # up is zeros: the same gradient
    (got2,) = torch.autograd.grad(adapted(x, torch.zeros(5, dtype=torch.int32, device=DEV)), x, dy)
    assert torch.equal(got2, got)


@pytest.mark.parametrize("m", [8, 200])
def test_a_refused_call_wrote_nothing(L, gpu_lib, m):
    """Autograd is not told of memory that a refused call did not write."""
    w = _weight(gpu_lib, 256, 256, "row", 0.73)
    dy = torch.randn((m, 256), device=DEV).to(torch.bfloat16)
    out = torch.zeros((m, 256), device=DEV)
    before = out._version
    for call in (lambda: L.linear_backward(dy, w, -1.0, out=out), lambda: L.linear_backward(dy, w._replace(scale=w.scale.cpu()), 0.73, out=out),
                 lambda: L.linear_backward(dy, w, 0.73, out=out, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    assert out._version == before and not out.any()
    L.linear_backward(dy, w, 0.73, out=out)
    assert out._version > before


@pytest.mark.parametrize("m,n,k", [(1, 33, 64), (8, 1000, 512), (64, 777, 128), (65, 2048, 256), (333, 1001, 768), (512, 96, 32),
                                   (513, 1001, 64), (600, 2048, 512), (700, 40, 512)])
@pytest.mark.parametrize("form", ["row", 32, "4b", "3b"])
def test_the_workspace_is_enough(L, gpu_lib, m, n, k, form):
    """What is asked for is all that is written, in every path and with every kind of padding."""
    w = _weight(gpu_lib, n, k, form, 0.73)
    dy = torch.randn((m, n), device=DEV).to(torch.bfloat16)
    need = L.linear_backward_workspace_bytes(m, n, k, 3 if form == "3b" else 4)
    held = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    got = L.linear_backward(dy, w, 0.73, out_dtype=torch.float32, workspace=held[:need])
    assert (held[need:] == 77).all()
    want = dy.double() @ gpu_lib.dequantize(w, 0.73).double()
    bound = (n + 64) * 2.0 ** -24 * (dy.double().abs() @ gpu_lib.dequantize(w, 0.73).double().abs())
    assert ((got.double() - want).abs() <= bound + 2.0 ** -24 * (want.abs() + bound)).all()
