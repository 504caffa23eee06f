"""The attention layer end to end on the GPU, and moving rows of the cache: a chain fed at
once equals the same tokens fed one by one, every branch of a tree equals that branch fed
as a chain, and an accepted path moved up serves the next token like a chain."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as AO
from w4a16_linear_amd import attention as A
from w4a16_linear_amd import module as M
from w4a16_linear_amd.attention_module import OPQAttention, token_slots

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _layer(seed=0, hidden=256, heads=4, kv=2, dim=64, quantize=True, **kw):
    torch.manual_seed(seed)
    layer = OPQAttention(hidden, heads, kv, dim, max_positions=512, **kw).to(DEV, torch.bfloat16)
    if quantize:
        assert M.replace_with_opq(layer) == ["qkv", "o"]
    return layer


def _pages(batch, per, seed=1):
    ids = np.random.default_rng(seed).permutation(batch * per).reshape(batch, per)
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def _close(a, b):
    """Two ways to one result: bfloat16 weights and results, in other orders (two roundings
    each of values up to the row's own size), through the output projection."""
    a, b = a.float(), b.float()
    assert (a - b).norm() <= 4 * 2.0 ** -8 * b.norm(), float((a - b).norm() / b.norm())


def test_layer_against_float64(gpu_lib):
    """The whole layer against its parts in float64, from the stored keys and values."""
    layer = _layer()
    batch, draft, page = 2, 5, 16
    cache = layer.new_cache(8, page, "fp8", device=DEV)
    table = _pages(batch, 4)
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    x = torch.randn(batch, draft, 256, device=DEV).bfloat16()
    y = layer(x, cache, table, lens)
    fused = layer.qkv(x).view(batch * draft, 8, 64)
    pos = torch.arange(draft, dtype=torch.int32, device=DEV).repeat(batch)
    turned = A.rotary(fused[:, :6].contiguous(), pos, layer.rope(x.device)).view(batch, draft, 6, 64)
    slots = token_slots(table, torch.arange(draft, dtype=torch.int32, device=DEV).expand(batch, draft), page)
    k, v = A.cache_read(cache, slots.reshape(-1), torch.float32)
    k, v = (t.double().cpu().numpy().reshape(batch, draft, 2, 64) for t in (k, v))
    q = turned[:, :, :4].double().cpu().numpy()
    seen = np.tril(np.ones((draft, draft), bool))
    out = np.stack([np.concatenate([AO.attention(q[b, :, 2 * h:2 * h + 2], k[b, :, h], v[b, :, h], 0, seen, 0.125)[0]
                                    for h in range(2)], 1) for b in range(batch)])
    ref = layer.o(torch.from_numpy(out).to(DEV, torch.bfloat16).view(batch, draft, 256))
    _close(y, ref)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_chain_equals_one_by_one(gpu_lib, fmt, layout):
    layer = _layer(3, layout=layout, rot=32)
    x = torch.randn(2, 20, 256, device=DEV).bfloat16()
    table = _pages(2, 3)
    at_once, steps = layer.new_cache(6, 16, fmt, device=DEV), layer.new_cache(6, 16, fmt, device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    y = layer(x, at_once, table, lens)
    one = torch.cat([layer(x[:, t:t + 1].contiguous(), steps, table, lens + t) for t in range(20)], 1)
    _close(one, y)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_tree_branches_and_accepting_one(gpu_lib, fmt):
    layer = _layer(5)
    batch, prefix, page = 2, 19, 16
    table = _pages(batch, 4)
    parents = torch.tensor([[-1, 0, 0, 1, 2, -1, 4], [-1, 0, 1, -1, 3, 3, 5]], dtype=torch.int32)
    draft = parents.shape[1]
    depth = torch.zeros_like(parents)
    for t in range(draft):
        for b in range(batch):
            depth[b, t] = 0 if parents[b, t] < 0 else depth[b, parents[b, t]] + 1
    mask, depths = A.tree_mask(parents).to(DEV), depth.to(DEV)
    first = torch.randn(batch, prefix, 256, device=DEV).bfloat16()
    x = torch.randn(batch, draft, 256, device=DEV).bfloat16()
    zero = torch.zeros(batch, dtype=torch.int32, device=DEV)
    lens = zero + prefix
    tree = layer.new_cache(8, page, fmt, device=DEV)
    layer(first, tree, table, zero)
    y = layer(x, tree, table, lens, mask=mask, depths=depths)
    paths = ([0, 2, 4, 6], [3, 5, 6])
    for b, path in enumerate(paths):
        chain = layer.new_cache(8, page, fmt, device=DEV)
        layer(first, chain, table, zero)
        c = layer(x[:, path].contiguous(), chain, table, lens)
        _close(y[b, path], c[b])
    # keep both paths; the next token then sees what the chain's next token sees
    kept = torch.tensor([[0, 2, 4, 6], [3, 5, 6, -1]], dtype=torch.int32, device=DEV)
    layer.accept(tree, table, lens, kept)
    after = lens + torch.tensor([4, 3], dtype=torch.int32, device=DEV)
    nxt = torch.randn(batch, 1, 256, device=DEV).bfloat16()
    got = layer(nxt, tree, table, after)
    for b, path in enumerate(paths):
        chain = layer.new_cache(8, page, fmt, device=DEV)
        layer(first, chain, table, zero)
        layer(x[:, path].contiguous(), chain, table, lens)
        want = layer(nxt, chain, table, lens + len(path))
        _close(got[b], want[b])


def test_counts_leave_padding_out(gpu_lib):
    layer = _layer(7)
    table = _pages(2, 2)
    x = torch.randn(2, 6, 256, device=DEV).bfloat16()
    counts = torch.tensor([6, 2], dtype=torch.int32, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    a, b = layer.new_cache(4, 16, "fp8", device=DEV), layer.new_cache(4, 16, "fp8", device=DEV)
    y = layer(x, a, table, zero, counts=counts)
    z = layer(x, b, table, zero)
    _close(y[0], z[0])
    _close(y[1, :2], z[1, :2])
    slots = token_slots(table, torch.arange(2, 6, dtype=torch.int32, device=DEV)[None].expand(2, 4), 16)
    assert not A.cache_read(a, slots[1].contiguous())[0].any()      # nothing written for padding


# ------------------------------------------------------------------ moving rows

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (128, 3, 32), (256, 2, 16)])
def test_move(gpu_lib, fmt, dim, heads, page):
    """Up to 128 moves with slots that are sources and destinations at once, and none-moves;
    the rows move bit for bit and the others stay."""
    pages, batch, count = 24, 2, 128
    cache = A.new_cache(pages, heads, page, dim, fmt, device=DEV)
    total = pages * page
    every = torch.arange(total, dtype=torch.int32, device=DEV)
    A.cache_write(cache, torch.randn(total, heads, dim, device=DEV), torch.randn(total, heads, dim, device=DEV), every)
    rng = np.random.default_rng(dim)
    half = total // 2
    src = np.stack([rng.integers(0, half, count), half + rng.integers(0, half, count)]).astype(np.int32)
    dst = np.stack([rng.permutation(half)[:count], half + rng.permutation(half)[:count]]).astype(np.int32)
    src[0, 5], dst[0, 9], src[1, 0], dst[1, 127] = -1, -1, total, 2 ** 31 - 1
    ref = [None if t is None else t.view(torch.uint8).cpu().numpy().copy() for t in cache[2:]]
    want = [None if r is None else r.copy() for r in ref]
    for b in range(batch):
        for f, t in zip(src[b], dst[b]):
            if 0 <= f < total and 0 <= t < total:
                for i, (r, w) in enumerate(zip(ref, want)):
                    if r is not None and i % 3 != 2:                # codes and signs: [pages, heads, page, bytes]
                        w[t // page, :, t % page] = r[f // page, :, f % page]
                    elif r is not None:                             # scales: [pages, heads, page * 4 bytes]
                        w[t // page, :, t % page * 4:t % page * 4 + 4] = r[f // page, :, f % page * 4:f % page * 4 + 4]
    A.cache_move(cache, torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV))
    for t, w in zip(cache[2:], want):
        assert t is None or np.array_equal(t.view(torch.uint8).cpu().numpy(), w)


def test_move_refusals_and_empty(gpu_lib):
    cache = A.new_cache(2, 2, 16, 64, "fp8", device=DEV)
    s = torch.zeros((1, 3), dtype=torch.int32, device=DEV)
    A.cache_move(cache, s[:, :0], s[:, :0])
    for a, b in ((s[0], s[0]), (s, s[:, :2]), (s.long(), s.long()), (s.cpu(), s), (s.expand(1, 3).repeat(1, 43), None)):
        with pytest.raises(ValueError):
            A.cache_move(cache, a, a if b is None else b)


def test_layer_refusals():
    for bad in (dict(heads=4, kv_heads=3, dim=64), dict(heads=4, dim=80)):
        with pytest.raises(ValueError):
            OPQAttention(256, **bad)


@pytest.mark.parametrize("bad", [2 ** 28, -2 ** 31, 2 ** 28 + 1, 4, -1])
def test_a_page_outside_the_cache_leaves_the_others_alone(gpu_lib, bad):
    """Page ids that wrap around to pages 0 and 1 in 32 bits, and ids just outside: nothing of
    another sequence is written over, by a forward or by accept."""
    layer = _layer(11)
    cache = layer.new_cache(4, 16, "fp8", device=DEV)
    good = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    layer(torch.randn(1, 32, 256, device=DEV).bfloat16(), cache, good, zero)
    before = [t.view(torch.uint8).clone() for t in cache[2:] if t is not None]
    table = torch.full((1, 2), bad, dtype=torch.int32, device=DEV)
    layer(torch.randn(1, 20, 256, device=DEV).bfloat16(), cache, table, zero)
    layer.accept(cache, table, zero, torch.tensor([[3, 5, 18]], dtype=torch.int32, device=DEV))
    mixed = torch.tensor([[0, bad]], dtype=torch.int32, device=DEV)
    layer.accept(cache, mixed, zero + 10, torch.tensor([[-1, 8, 9]], dtype=torch.int32, device=DEV))
    for t, b in zip((t for t in cache[2:] if t is not None), before):
        assert torch.equal(t.view(torch.uint8), b)


def test_first_calls_on_two_streams(gpu_lib):
    """The first call makes the rotary table; a call on another stream right behind it reads
    the finished one, however busy the first stream is."""
    x = torch.randn(2, 9, 256, device=DEV).bfloat16()
    table = _pages(2, 1)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    ref_layer = _layer(13)
    ref = ref_layer(x, ref_layer.new_cache(2, 16, "fp8", device=DEV), table, zero)
    layer = _layer(13)
    caches = [layer.new_cache(2, 16, "fp8", device=DEV) for _ in range(2)]
    big = torch.randn(4096, 4096, device=DEV).bfloat16()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(first):
        for _ in range(100):
            big @ big
        a = layer(x, caches[0], table, zero)
    with torch.cuda.stream(second):
        b = layer(x, caches[1], table, zero)
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    assert layer.rope(x.device) is layer.rope("cuda")


def test_layer_in_a_graph(gpu_lib):
    """A capture that would have to make the table is refused; once it is there the layer's
    step is captured and replayed, each replay equal to the eager call and following lengths
    changed in place."""
    layer = _layer(17)
    x = torch.randn(2, 1, 256, device=DEV).bfloat16()
    first = torch.randn(2, 20, 256, device=DEV).bfloat16()
    table = _pages(2, 4)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    cache = layer.new_cache(8, 16, "opq4", device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(RuntimeError, match="rotary table"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            layer(x, cache, table, zero)
    layer(first, cache, table, zero)
    lens = zero + 20
    want = [layer(x, cache, table, zero + n) for n in (20, 21, 20, 21)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y = layer(x, cache, table, lens, max_len=48)
    for i in range(4):
        y.zero_()
        lens.copy_(zero + 20 + i % 2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        layer(first, layer.new_cache(8, 16, "opq4", device=DEV), table, zero)


def test_a_refused_forward_writes_nothing(gpu_lib):
    layer = _layer(19)
    cache = layer.new_cache(2, 16, "fp8", device=DEV)
    x = torch.randn(1, 3, 256, device=DEV).bfloat16()
    args = dict(x=x, cache=cache, page_table=_pages(1, 2), lens=torch.zeros(1, dtype=torch.int32, device=DEV))
    for bad in (dict(x=x.float()), dict(page_table=_pages(1, 2).long()), dict(max_len=33),
                dict(counts=torch.ones(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            layer(**{**args, **bad})
    assert not any(t.view(torch.uint8).any() for t in cache[2:] if t is not None)
    layer(**args)
    assert cache.k_scale.any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("dim,page", [(128, 64), (256, 256)])
def test_prompt_at_once_equals_in_chunks(gpu_lib, fmt, dim, page):
    """A prompt of 400 tokens at once, in three chunks of odd lengths, and its last token alone."""
    layer = _layer(23, hidden=512, heads=4, kv=2, dim=dim)
    x = torch.randn(2, 400, 512, device=DEV).bfloat16()
    per = -(-400 // page)
    table = _pages(2, per)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    at_once, chunks = (layer.new_cache(2 * per, page, fmt, device=DEV) for _ in range(2))
    y = layer(x, at_once, table, zero)
    parts = [layer(x[:, a:b].contiguous(), chunks, table, zero + a, max_len=a) for a, b in ((0, 129), (129, 399), (399, 400))]
    _close(torch.cat(parts, 1), y)


def test_rope_by_any_name(gpu_lib):
    """One table a device, whether it is named by a tensor's device, an index or without one."""
    layer = _layer(29, quantize=False)
    table = layer.rope("cuda")
    here = torch.cuda.current_device()
    assert all(layer.rope(d) is table for d in ("cuda", f"cuda:{here}", torch.device("cuda"), torch.device("cuda", here),
                                                table.device))


def test_no_tokens(gpu_lib):
    """A step without tokens, and one without sequences: nothing written, empty results."""
    layer = _layer(31)
    cache = layer.new_cache(2, 16, "fp8", device=DEV)
    x = torch.randn(1, 3, 256, device=DEV).bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert layer(x[:, :0], cache, _pages(1, 2), zero).shape == (1, 0, 256)
    assert layer(x[:0], cache, _pages(1, 2)[:0], zero[:0]).shape == (0, 3, 256)
    counts = zero.clone()
    assert layer(x[:, :1], cache, _pages(1, 2), zero, counts=counts).shape == (1, 1, 256)
    assert not any(t.view(torch.uint8).any() for t in cache[2:] if t is not None)
