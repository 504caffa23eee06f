"""What the adapters' sums hold: bfloat16 results that are the float32 ones rounded."""
import pytest
import torch

from test_gpu_adapters import DEV, _gen, _index, _stack

pytestmark = pytest.mark.gpu

# one launch; a wide block of tokens; one adapter's and mixed tokens of several blocks, each width of ranks
SIZES = [(1, 256, 264, 8, 3), (40, 256, 264, 16, 3), (50, 2048, 1032, 32, 5), (64, 256, 264, 64, 3), (300, 256, 1032, 8, 2),
         (300, 128, 520, 40, 5), (200, 128, 264, 128, 3)]


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


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
