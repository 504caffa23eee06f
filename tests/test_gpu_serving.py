"""A server's step with everything in it: adapters beside quantized projections, drafted tokens
through the paged cache, their verification, what is kept of them, rows forked and dropped, pages
drawn together.  After every step each row answers as it does when its tokens are run afresh."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HIDDEN, HEADS, VOCAB, DRAFT = 256, 4, 97, 5


@pytest.fixture(scope="module")
def A(gpu_lib):
    from w4a16_linear_amd import attention
    attention.load()
    return attention


def _model(seed=0):
    from w4a16_linear_amd.attention_module import OPQAttention
    from w4a16_linear_amd.module import add_adapters, replace_with_opq
    torch.manual_seed(seed)
    layer = OPQAttention(HIDDEN, heads=HEADS, kv_heads=2, max_positions=1024).to(torch.bfloat16).to(DEV)
    replace_with_opq(layer)
    assert add_adapters(layer, 3, 8) == ["qkv", "o"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    with torch.no_grad():
        for mod in (layer.qkv, layer.o):
            mod.up.copy_(torch.randn(mod.up.shape, generator=g, device=DEV) * 0.2)
    embed = torch.randn((VOCAB, HIDDEN), generator=g, device=DEV).to(torch.bfloat16)
    head = torch.randn((HIDDEN, VOCAB), generator=g, device=DEV) * 0.3
    return layer, embed, head


@torch.no_grad()
def test_a_serving_loop(A):
    from w4a16_linear_amd.attention_module import PagedSequences
    from w4a16_linear_amd.module import use_adapters
    layer, embed, head = _model()
    rows, columns, page, pages = 6, 12, 16, 80
    cache = layer.new_cache(pages, page, "bf16")
    seqs = PagedSequences(rows, columns, pages, page)
    rng = np.random.default_rng(0)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    adapter = torch.tensor([0, 1, -1, 2, 1, 0], dtype=torch.int32, device=DEV)
    tokens = [[] for _ in range(rows)]                       # what is cached, row by row
    root = torch.from_numpy(rng.integers(0, VOCAB, rows).astype(np.int32)).to(DEV)

    def probabilities(y):
        return torch.softmax(y.float() @ head, -1)

    for step in range(8):
        draft = torch.from_numpy(rng.integers(0, VOCAB, (rows, DRAFT)).astype(np.int32)).to(DEV)
        draft[:, 0] = root
        parents = np.tile(np.arange(-1, DRAFT - 1), (rows, 1))
        if step % 2:                                         # trees: two candidates under most nodes
            parents[:, 2:] = np.maximum(0, (np.arange(2, DRAFT) - 1) // 2)
        par = torch.from_numpy(parents.astype(np.int32))
        depth = np.zeros((rows, DRAFT), np.int32)
        for i in range(1, DRAFT):
            depth[:, i] = depth[np.arange(rows), parents[:, i]] + 1
        mask, depths = A.tree_mask(par).to(DEV), torch.from_numpy(depth).to(DEV)
        assert seqs.room(DRAFT).tolist() == [0]
        use_adapters(layer, adapter)
        y = layer(embed[draft.long()], cache, seqs.page_table, seqs.lens, mask=mask, depths=depths)
        p = probabilities(y)
        if step < 2:                                         # make sure that drafts are kept at times
            p = torch.where(torch.arange(VOCAB, device=DEV) == draft.roll(-1, 1)[..., None], p + 2.0, p)
            p = p / p.sum(-1, keepdim=True)
        u = torch.rand((rows, DRAFT), generator=g, device=DEV)
        kept, count, following = A.verify_drafts(p, draft, u, parents=par.to(DEV))
        seqs.accept([cache], kept, count)
        for b in range(rows):
            tokens[b] += [int(draft[b, i]) for i in kept[b].tolist() if i >= 0]
        assert seqs.lens.tolist() == [len(t) for t in tokens] and (following >= 0).all()
        root = following
        if step % 3 == 1:                                    # beams: rows go on twice, one is dropped
            order = rng.integers(0, rows, rows)
            order[rng.integers(0, rows)] = -1
            where = torch.from_numpy(order.astype(np.int32)).to(DEV)
            assert seqs.fork([cache], where).tolist() == [0]
            tokens = [list(tokens[a]) if a >= 0 else [] for a in order]
            pick = where.clamp_min(0).long()
            root, adapter = root[pick], adapter[pick]
        if step % 4 == 2:
            used = int(seqs.compact([cache]))
            assert int(seqs.page_table.max()) < used
        # every row as if its tokens were run afresh, in one call, in a cache of its own
        longest = max(len(t) for t in tokens) + 1
        fresh = layer.new_cache(rows * columns, page, "bf16")
        table = torch.arange(rows * columns, dtype=torch.int32, device=DEV).view(rows, columns)
        ids = torch.zeros((rows, longest), dtype=torch.long, device=DEV)
        for b in range(rows):
            ids[b, :len(tokens[b]) + 1] = torch.tensor(tokens[b] + [int(root[b])], device=DEV)
        use_adapters(layer, adapter)
        whole = layer(embed[ids], fresh, table, torch.zeros(rows, dtype=torch.int32, device=DEV))
        assert seqs.room(1).tolist() == [0]
        now = layer(embed[root.long()][:, None], cache, seqs.page_table, seqs.lens)
        want = whole[torch.arange(rows, device=DEV), seqs.lens.long()]
        # bfloat16 activations through two projections and the attention: a few roundings of 2^-8 of
        # values of the row's own size
        err = (now[:, 0].float() - want.float()).abs().amax(1)
        assert (err <= 2.0 ** -5 * want.float().abs().amax(1)).all(), (step, err.tolist())
        seqs.room(0)


def test_one_graph_of_a_step(A):
    """Verification, accepted rows moved, rows forked, resized and compacted, pages copied: captured
    together, replayed on new contents, against eager calls."""
    rng = np.random.default_rng(2)
    rows, columns, page, pages, draft, vocab = 8, 10, 16, 120, 6, 700
    caches = [A.new_cache(pages, 2, page, 64, "fp8") for _ in range(2)]
    for t in (*caches[0][2:], *caches[1][2:]):
        if t is not None:
            t.view(torch.uint8).random_(0, 100)

    def state():
        lens = rng.integers(0, columns * page - draft, rows)
        table = np.full((rows, columns), -1)
        ids = rng.permutation(pages)
        at = 0
        for i in range(rows):
            n = -(-(lens[i] + draft) // page)
            table[i, :n] = ids[at:at + n]
            at += n
        p = torch.softmax(torch.randn((rows, draft, vocab), device=DEV) * 2, -1)
        q = torch.softmax(torch.randn((rows, draft - 1, vocab), device=DEV) * 2, -1)
        return [torch.from_numpy(table.astype(np.int32)).to(DEV), torch.from_numpy(lens.astype(np.int32)).to(DEV),
                torch.from_numpy(rng.integers(0, vocab, (rows, draft)).astype(np.int32)).to(DEV), p, q,
                torch.rand((rows, draft), device=DEV), torch.from_numpy(rng.integers(-1, rows, rows).astype(np.int32)).to(DEV)]

    def step(cache, table, lens, tokens, p, q, u, parents):
        kept, count, nxt = A.verify_drafts(p, tokens, u, draft_probs=q)
        table, missing = A.pages_resize(table, lens + count, pages, page)
        table, lens2, src, dst, lost = A.pages_fork(table, lens + count, parents, pages, page)
        A.cache_copy_pages(cache, src, dst)
        table, src2, dst2, used = A.pages_compact(table, pages)
        A.cache_copy_pages(cache, src2, dst2)
        return kept, count, nxt, table, missing, lens2, src, dst, lost, src2, dst2, used

    held = state()
    start = [None if t is None else t.clone() for t in caches[0][2:]]

    def reset(cache):
        for t, v in zip(cache[2:], start):
            if t is not None:
                t.view(torch.uint8).copy_(v.view(torch.uint8))

    step(caches[0], *held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(caches[0], *held)
    for _ in range(4):
        for t, v in zip(held, state()):
            t.copy_(v)
        reset(caches[0])
        reset(caches[1])
        graph.replay()
        torch.cuda.synchronize()
        want = step(caches[1], *held)
        torch.cuda.synchronize()
        assert all(torch.equal(r, e) for r, e in zip(res, want))
        for a, b in zip(caches[0][2:], caches[1][2:]):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_sequences_refuse_other_caches(A):
    from w4a16_linear_amd.attention_module import PagedSequences
    seqs = PagedSequences(2, 3, 8, 16)
    for cache in (A.new_cache(9, 1, 16, 64), A.new_cache(8, 1, 32, 64)):
        with pytest.raises(ValueError, match="pages"):
            seqs.fork([cache], torch.zeros(2, dtype=torch.int32, device=DEV))
    assert seqs.room(100).tolist() == [0] and seqs.room(torch.tensor([0, 17], dtype=torch.int32, device=DEV)).tolist() == [0]
    small = PagedSequences(2, 9, 4, 16)
    assert small.room(64).tolist() == [4] and small.page_table[1].max() == -1
