"""Adapters in the saved form: what save_opq writes of an adapted model, load_opq gives back, to a
skeleton, to the model before it was quantized or adapted, and to an adapted one (no GPU needed)."""
import json

import pytest
import torch
from safetensors import safe_open
from torch import nn

from w4a16_linear_amd.module import AdaptedLinear, OPQLinear, add_adapters, load_opq, save_opq


class Net(nn.Module):
    def __init__(self, kind=nn.Linear):
        super().__init__()
        self.a = kind(64, 64)
        self.again = self.a
        self.b = nn.Sequential(kind(64, 24), kind(64, 20))   # 20: no multiple of 8, so not adapted


def _filled(seed=0):
    g = torch.Generator().manual_seed(seed)
    m = Net(OPQLinear)
    for t in m.buffers():
        if t.dtype == torch.int32:
            t.copy_(torch.randint(-2 ** 31, 2 ** 31, t.shape, generator=g, dtype=torch.int64).to(torch.int32))
        else:
            t.copy_(torch.rand(t.shape, generator=g))
    return m


def _adapted(seed=0, count=3, rank=5):
    m = _filled(seed)
    assert add_adapters(m, count, rank) == ["a", "again", "b.0"]
    g = torch.Generator().manual_seed(seed + 1)
    with torch.no_grad():
        for layer in (m.a, m.b[0]):
            layer.down[:, :rank] = torch.randn(layer.down[:, :rank].shape, generator=g).bfloat16()
            layer.up[:, :rank] = torch.randn(layer.up[:, :rank].shape, generator=g).bfloat16()
            layer.scale.copy_(torch.rand(count, generator=g))
    return m


def _same(a, b):
    x, y = a.state_dict(), b.state_dict()
    assert list(x) == list(y)
    for k in x:
        assert x[k].dtype == y[k].dtype and torch.equal(x[k], y[k]), k


@pytest.mark.parametrize("into", ["skeleton", "quantized", "adapted", "adapted otherwise"])
def test_an_adapted_model_comes_back(tmp_path, into):
    path = str(tmp_path / "m.safetensors")
    m = _adapted()
    assert save_opq(m, path) == ["a", "b.0", "b.1"]
    other = {"skeleton": Net, "quantized": lambda: _filled(7), "adapted": lambda: _adapted(7),
             "adapted otherwise": lambda: _adapted(7, count=1, rank=16)}[into]()
    assert load_opq(other, path) == ["a", "b.0", "b.1"]
    _same(m, other)
    assert other.a is other.again and isinstance(other.a, AdaptedLinear) and isinstance(other.b[1], OPQLinear)
    assert other.a.rank == 5 and other.a.down.requires_grad and other.a.up.requires_grad


def test_a_file_without_adapters_fills_the_base(tmp_path):
    """The projections of an adapted model are replaced, its adapters stay."""
    path = str(tmp_path / "m.safetensors")
    base, m = _filled(3), _adapted(5)
    save_opq(base, path)
    kept = {k: v.clone() for k, v in m.state_dict().items()}
    assert load_opq(m, path) == ["a", "b.0", "b.1"]
    assert isinstance(m.a, AdaptedLinear) and m.a is m.again and isinstance(m.a.base, OPQLinear)
    for k, v in m.state_dict().items():
        if k.rsplit(".", 1)[1] in ("down", "up", "scale"):
            assert torch.equal(v, kept[k])
        else:
            assert torch.equal(v, base.state_dict()[k.replace(".base", "")]), k


def test_files_of_either_kind_say_which(tmp_path):
    """A file without adapters is as it was; one with them is of another format, which a reader that
    would leave them out refuses."""
    path = str(tmp_path / "m.safetensors")
    for m, fmt in ((_filled(), "opq-int4/1"), (_adapted(), "opq-int4/2")):
        save_opq(m, path)
        with safe_open(path, framework="pt") as f:
            meta = json.loads(f.metadata()["opq"])
            assert meta["format"] == fmt
            codes, adapters = {"a.packed", "a.sign_packed", "a.mx", "a.bias"}, {"a.down", "a.up", "a.scale"}
            assert {k for k in f.keys() if k.startswith("a.")} == (codes | adapters if fmt.endswith("2") else codes)
            assert not any(".base." in k for k in f.keys())


def test_parameters_of_the_same_shape_stay_the_ones_an_optimizer_knows(tmp_path):
    path = str(tmp_path / "m.safetensors")
    m, other = _adapted(), _adapted(7)
    save_opq(m, path)
    layer, down, index = other.a, other.a.down, torch.zeros(3, dtype=torch.int32)
    layer.index = index
    load_opq(other, path)
    assert other.a is layer and layer.down is down and layer.index is index
    _same(m, other)


def test_names_of_the_inner_layer(tmp_path):
    """A file that names an adapted layer's projection itself (`a.base`) still fills it."""
    path = str(tmp_path / "m.safetensors")

    class Inner(nn.Module):
        def __init__(self, layer):
            super().__init__()
            self.base = layer

    holder = nn.Module()
    holder.a = Inner(_filled(9).a)
    assert save_opq(holder, path) == ["a.base"]
    m = _adapted(5)
    assert load_opq(m, path) == ["a.base"]
    assert isinstance(m.a, AdaptedLinear) and torch.equal(m.a.base.packed, holder.a.base.packed)


def test_what_does_not_fit_is_refused(tmp_path):
    path = str(tmp_path / "m.safetensors")
    m = _adapted()
    save_opq(m, path)
    other = Net()
    other.b[0] = nn.Linear(64, 32)
    with pytest.raises(ValueError, match="24x64"):
        load_opq(other, path)
    other = Net()
    other.a = other.again = nn.Identity()
    with pytest.raises(ValueError, match="not a Linear"):
        load_opq(other, path)
