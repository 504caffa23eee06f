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
                                   (257, 96, 512), (300, 520, 1024), (333, 3840, 512), (1024, 200, 256)])
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
