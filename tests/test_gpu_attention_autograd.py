"""The attention side's calls and autograd: only apply_rotary is followed; the others refuse
tensors that require grad, and tell autograd of memory that they write."""
import pytest
import torch

from w4a16_linear_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _parts():
    x = torch.randn(3, 2, 64, device=DEV).bfloat16()
    index = torch.arange(3, dtype=torch.int32, device=DEV)
    cache = A.new_cache(2, 2, 16, 64, "opq4", device=DEV)
    A.cache_write(cache, x, x, index)
    return x, index, A.rotary_table(A.rotary_frequencies(64), 8, DEV), cache


def _calls():
    """(name, the call with one tensor t in place) for every tensor a gradient could flow to."""
    x, index, table, cache = _parts()
    q, lens = x[:1].view(1, 1, 2, 64), index[:1]
    pages = index[None, :2]
    return {
        "rotary x": (x, lambda t: A.rotary(t, index, table)),
        "rotary table": (table, lambda t: A.rotary(x, index, t)),
        "rotary out": (torch.empty_like(x), lambda t: A.rotary(x, index, table, out=t)),
        "rotary_backward": (x, lambda t: A.rotary_backward(t, index, table)),
        "apply_rotary table": (table, lambda t: A.apply_rotary(x, index, t)),
        "cache_write k": (x, lambda t: A.cache_write(cache, t, x, index)),
        "cache_write v": (x, lambda t: A.cache_write(cache, x, t, index)),
        "cache_read out": (torch.empty_like(x), lambda t: A.cache_read(cache, index, out=(t, torch.empty_like(x)))),
        "attention q": (q, lambda t: A.tree_attention(t, cache, pages, lens)),
        "attention out": (torch.empty_like(q), lambda t: A.tree_attention(q, cache, pages, lens, out=t)),
    }


NAMES = ["rotary x", "rotary table", "rotary out", "rotary_backward", "apply_rotary table", "cache_write k",
         "cache_write v", "cache_read out", "attention q", "attention out"]


@pytest.mark.parametrize("name", NAMES)
def test_lost_gradients_are_refused(gpu_lib, name):
    t, call = _calls()[name]
    call(t)
    t = t.detach().clone().requires_grad_()
    with pytest.raises(RuntimeError, match="requires grad"):
        call(t)
    with torch.no_grad():
        call(t)
    with torch.inference_mode():
        call(t)
    call(t.detach())


def test_written_memory_is_known_to_autograd(gpu_lib):
    """A tensor that a product saved for its backward, then written in place: the backward
    says so, and does not use the new values."""
    x, index, table, cache = _parts()
    q = x[:1].view(1, 1, 2, 64)
    lens, pages = index[:1], index[None, :2]
    writes = [(x.clone(), lambda t: A.rotary(t, index, table, out=t)),
              (x.clone(), lambda t: A.cache_read(cache, index, out=(t, torch.empty_like(x)))),
              (q.clone(), lambda t: A.tree_attention(q, cache, pages, lens, out=t)),
              (cache.k_scale, lambda t: A.cache_write(cache, x, x, index)),
              (cache.v_scale, lambda t: A.cache_move(cache, index[None], index[None]))]
    for t, write in writes:
        w = torch.ones_like(t, requires_grad=True)
        y = w * t
        write(t)
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.sum().backward()


def test_inference_tensors_are_written_as_before(gpu_lib):
    with torch.inference_mode():
        x, index, table, cache = _parts()
        out = torch.empty_like(x)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            A.rotary(x, index, table, out=out)
            A.cache_write(cache, x, x, index)
            A.cache_read(cache, index, out=(out, torch.empty_like(x)))
    assert torch.isfinite(out).all()
