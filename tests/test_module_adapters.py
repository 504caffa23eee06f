"""The adapters' front end without a GPU: construction, filling, conversion, refusals."""
import pytest
import torch
from torch import nn

from w4a16_linear_amd.module import AdaptedLinear, OPQLinear, add_adapters, use_adapters


def test_a_stack_is_padded_and_filled():
    layer = AdaptedLinear(OPQLinear(64, 24), 3, 5, scale=2.0)
    assert layer.down.shape == (3, 8, 64) and layer.up.shape == (3, 8, 24) and layer.scale.tolist() == [2.0] * 3
    assert layer.down.dtype == layer.up.dtype == torch.bfloat16 and not layer.up.any() and not layer.down[:, 5:].any()
    assert {n for n, p in layer.named_parameters() if p.requires_grad} == {"down", "up"}
    down, up = torch.randn(4, 64).bfloat16(), torch.randn(24, 4).bfloat16()
    layer.set_adapter(1, down, up, 0.5)
    assert torch.equal(layer.down[1, :4], down) and torch.equal(layer.up[1, :4], up.t()) and not layer.down[1, 4:].any()
    assert layer.scale.tolist() == [2.0, 0.5, 2.0]
    for args in ((3, down, up), (-1, down, up), (0, down[:, :32], up), (0, torch.zeros(6, 64), torch.zeros(24, 6)),
                 (0, down, up.t())):
        with pytest.raises(ValueError):
            layer.set_adapter(*args)


@pytest.mark.parametrize("args", [(OPQLinear(64, 20), 1, 8), (OPQLinear(64, 24), 0, 8), (OPQLinear(64, 24), 1, 0),
                                  (OPQLinear(64, 24), 1, 129), (nn.Linear(64, 24), 1, 8)])
def test_refusals(args):
    with pytest.raises(ValueError):
        AdaptedLinear(*args)


class Block(nn.Module):
    def __init__(self):
        super().__init__()
        self.a = OPQLinear(64, 64)
        self.b = self.a                       # the same layer twice
        self.c = nn.Sequential(OPQLinear(32, 20), OPQLinear(32, 40), nn.Linear(8, 8))
        self.skipped = OPQLinear(64, 64)


def test_add_and_use_adapters():
    m = Block()
    assert add_adapters(m, 2, 4, skip=("skipped",)) == ["a", "b", "c.1"]
    assert m.a is m.b and isinstance(m.a, AdaptedLinear) and isinstance(m.c[0], OPQLinear) and isinstance(m.skipped, OPQLinear)
    assert add_adapters(m, 2, 4, skip=("skipped",)) == []          # once is enough
    index = torch.zeros(3, dtype=torch.int32)
    use_adapters(m, index)
    assert m.a.index is index and m.c[1].index is index
    use_adapters(m, None)
    assert m.a.index is None
    assert {"a.base.packed", "a.down", "a.up", "a.scale"} <= set(m.state_dict())


def test_forward_refuses():
    layer = AdaptedLinear(OPQLinear(64, 24), 3, 8)
    x = torch.zeros(2, 5, 64)
    for index in (torch.zeros(2, 5), torch.zeros(5, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32),
                  torch.zeros(2, 5, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="index"):
            layer(x, index)
    for bad in (x[..., :32], x.half()):
        with pytest.raises(ValueError):
            layer(bad, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):                   # no CPU path
        layer(x, torch.zeros(2, dtype=torch.int32))
