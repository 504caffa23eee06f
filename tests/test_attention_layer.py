"""CPU tests of the attention layer's host parts: cache slots of positions, what a forward
refuses before anything is enqueued."""
import numpy as np
import pytest
import torch

from w4a16_linear_amd.attention_module import OPQAttention, token_slots


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------ slots

@pytest.mark.parametrize("page", [16, 64, 1024])
def test_slots_equal_their_definition(page):
    rng = np.random.default_rng(page)
    pages = 50
    table = rng.permutation(pages)[:24].reshape(3, 8).astype(np.int32)
    table[1, 2], table[2, 0], table[0, 7] = -1, pages, 2 ** 31 - 1
    pos = rng.integers(-page, 9 * page, (3, 200)).astype(np.int32)
    want = np.full(pos.shape, -1)
    for b in range(3):
        for i, p in enumerate(pos[b]):
            if 0 <= p < 8 * page and 0 <= table[b, p // page] < pages:
                want[b, i] = int(table[b, p // page]) * page + p % page
    got = token_slots(torch.from_numpy(table), torch.from_numpy(pos), page, pages)
    assert got.dtype == torch.int32 and np.array_equal(got.numpy(), want)


@pytest.mark.parametrize("pages", [None, 100])
@pytest.mark.parametrize("page,ids", [(64, 2 ** 26), (64, -2 ** 31), (64, 2 ** 26 + 3), (64, 2 ** 25), (64, 2 ** 31 - 1),
                                      (1024, 2 ** 22), (1024, -2 ** 31 + 5), (1024, 2 ** 21), (16, 2 ** 28 + 1), (16, -1)])
def test_a_page_id_outside_every_cache_names_no_slot(page, ids, pages):
    """Also where id * page + offset wraps around to a small number in 32 bits; a cache holds
    fewer than 2^31 tokens, so an id of 2^31 / page or more is outside whatever its size."""
    pos = _i32([[0, 1, page - 1, page, page + 1, 3 * page - 1]])
    got = token_slots(_i32([[ids, ids, ids]]), pos, page, pages)
    assert (got == -1).all()


def test_no_pages_no_slots():
    """A page table without columns, and a cache without pages: nothing to look up."""
    pos = _i32([[-1, 0, 5], [0, 70, 2 ** 31 - 1]])
    assert (token_slots(torch.zeros((2, 0), dtype=torch.int32), pos, 64) == -1).all()
    assert (token_slots(_i32([[-1, 0], [0, 1]]), pos, 64, 0) == -1).all()
    assert token_slots(torch.zeros((2, 0), dtype=torch.int32), pos[:, :0], 64).shape == (2, 0)
    assert token_slots(torch.zeros((0, 3), dtype=torch.int32), pos[:0], 64).shape == (0, 3)


# ------------------------------------------------------------------ refusals

def _call(**kw):
    """A forward with everything in order but what kw says, on the CPU: in order it gets as
    far as the rotary table, which needs the GPU."""
    layer = OPQAttention(128, 2, 1, 64, max_positions=64).to(torch.bfloat16)
    args = dict(x=torch.zeros(2, 3, 128, dtype=torch.bfloat16), cache=layer.new_cache(4, 16, "fp8", device="cpu"),
                page_table=_i32([[0, 1], [2, 3]]), lens=_i32([0, 5]))
    with torch.no_grad():
        layer(**{**args, **kw})


def test_in_order_reaches_the_gpu():
    tree = dict(mask=torch.zeros((2, 3, 1), dtype=torch.int32), depths=torch.zeros((2, 3), dtype=torch.int32))
    for kw in (dict(), tree, dict(tree, mask=tree["mask"][0]), dict(counts=_i32([3, 0])), dict(max_len=0), dict(max_len=32)):
        with pytest.raises(ValueError, match="CUDA"):
            _call(**kw)


def test_a_mask_needs_depths():
    with pytest.raises(ValueError, match="depths"):
        _call(mask=torch.zeros((2, 3, 1), dtype=torch.int32))


_TREE = dict(mask=torch.zeros((2, 3, 1), dtype=torch.int32), depths=torch.zeros((2, 3), dtype=torch.int32))


@pytest.mark.parametrize("name,bad", [
    ("x", dict(x=torch.zeros(2, 3, 128))), ("x", dict(x=torch.zeros(2, 3, 128, dtype=torch.float16))),
    ("x", dict(x=torch.zeros(3, 128, dtype=torch.bfloat16))), ("x", dict(x=torch.zeros(2, 3, 64, dtype=torch.bfloat16))),
    ("page_table", dict(page_table=torch.zeros((2, 2), dtype=torch.int64))),
    ("page_table", dict(page_table=_i32([[0, 1]]))), ("page_table", dict(page_table=_i32([0, 1]))),
    ("contiguous", dict(page_table=_i32([[0, 1, 2], [1, 2, 3]])[:, :2])),
    ("lens", dict(lens=torch.zeros(2, dtype=torch.int64))), ("lens", dict(lens=_i32([0]))),
    ("mask", dict(_TREE, mask=_TREE["mask"].long())), ("mask", dict(_TREE, mask=_TREE["mask"][:, :2])),
    ("mask", dict(_TREE, mask=_TREE["mask"][:1])), ("depths", dict(_TREE, depths=_TREE["depths"].long())),
    ("depths", dict(_TREE, depths=_TREE["depths"][:, :2])), ("counts", dict(counts=_i32([1]))),
    ("counts", dict(counts=torch.ones(2))), ("max_len", dict(max_len=33)), ("max_len", dict(max_len=-1)),
    ("heads", dict(cache=OPQAttention(128, 2, 2, 64).new_cache(4, 16, "fp8", device="cpu"))),
    ("heads", dict(cache=OPQAttention(128, 2, 1, 128).new_cache(4, 16, "fp8", device="cpu")))])
def test_refused_before_anything_is_enqueued(name, bad):
    """What a later call of the forward refuses is refused before an earlier one has written
    to the cache: here, before the GPU is asked for at all."""
    with pytest.raises(ValueError, match=name) as e:
        _call(**bad)
    assert "CUDA" not in str(e.value)


def test_lost_gradients_are_refused():
    """x or the weights of qkv would get no gradient: an error instead, unless none is asked for."""
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16)

    def call(layer, x):
        layer(x, layer.new_cache(1, 16, "fp8", device="cpu"), _i32([[0]]), _i32([0]))

    layer = OPQAttention(128, 2, 1, 64, max_positions=64).to(torch.bfloat16)
    with pytest.raises(RuntimeError, match="gradients"):
        call(layer, x)
    for quiet in (torch.no_grad, torch.inference_mode):
        with quiet(), pytest.raises(ValueError, match="CUDA"):
            call(layer, x)
    layer.qkv.requires_grad_(False)
    with pytest.raises(ValueError, match="CUDA"):
        call(layer, x)
    with pytest.raises(RuntimeError, match="gradients"):
        call(layer, x.requires_grad_())
