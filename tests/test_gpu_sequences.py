"""PagedSequences when pages run out: a row never counts a token that no page holds, and what a
row lost stays known until its caller says otherwise."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def A(gpu_lib):
    from w4a16_linear_amd import attention
    attention.load()
    return attention


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _filled(A, pages, rows, columns, lens, page=16):
    """Rows of the given lengths, every stored token's scale its row and position."""
    from w4a16_linear_amd.attention_module import PagedSequences, token_slots
    seqs = PagedSequences(rows, columns, pages, page)
    cache = A.new_cache(pages, 1, page, 64, "fp8")
    assert seqs.room(lens).tolist() == [0]
    seqs.lens = lens
    at = torch.arange(columns * page, dtype=torch.int32, device=DEV).expand(rows, -1)
    slots = token_slots(seqs.page_table, at, page, pages)
    mark = 1000.0 * (torch.arange(rows, device=DEV)[:, None] + 1) + at
    for t in (cache.k_scale, cache.v_scale):
        t.zero_()
        t.view(-1)[slots[slots >= 0].long()] = mark[slots >= 0].float()
    return seqs, cache


def _held(seqs, cache, row):
    """The marks of a row's tokens, as the cache holds them."""
    from w4a16_linear_amd.attention_module import token_slots
    n = int(seqs.lens[row])
    slots = token_slots(seqs.page_table, torch.arange(n, dtype=torch.int32, device=DEV).expand(seqs.page_table.shape[0], -1),
                        seqs.page, seqs.pages)[row]
    assert (slots >= 0).all()
    return cache.k_scale.view(-1)[slots.long()].tolist()


def test_a_fork_without_pages_keeps_what_it_has(A):
    seqs, cache = _filled(A, pages=2, rows=3, columns=2, lens=_ints(20, 0, 0))
    assert seqs.lost.tolist() == [0, 0, 0]
    assert seqs.fork([cache], _ints(0, 0, -1)).tolist() == [1]
    assert seqs.lens.tolist() == [20, 16, 0] and seqs.lost.tolist() == [0, 4, 0]
    assert _held(seqs, cache, 1) == [1000.0 + i for i in range(16)]
    # a page comes free: the row takes it for new tokens, not for those it lost
    assert seqs.fork([cache], _ints(-1, 1, -1)).tolist() == [0]
    assert seqs.lens.tolist() == [0, 16, 0] and seqs.lost.tolist() == [0, 4, 0]
    assert seqs.room(_ints(0, 1, 0)).tolist() == [0]
    assert seqs.lens.tolist() == [0, 16, 0] and seqs.lost.tolist() == [0, 4, 0]
    assert _held(seqs, cache, 1) == [1000.0 + i for i in range(16)]
    # what is lost follows the forks, ends with the row, and is the caller's to clear
    assert seqs.fork([cache], _ints(1, 1, 0)).tolist() == [0]
    assert seqs.lost.tolist() == [4, 4, 0]
    seqs.lost.zero_()
    seqs.room(0)
    assert seqs.lost.tolist() == [0, 0, 0]


@pytest.mark.parametrize("kept,count,lens,lost", [(list(range(12)), 12, 16, 6), ([0, 8, -1], 2, 11, 1), ([0, 3, -1], 2, 12, 0),
                                                  ([-1, -1], 0, 10, 0)])
@pytest.mark.parametrize("pages,columns", [(1, 4), (4, 1)])   # no page left, no column left
def test_tokens_that_no_page_took_are_not_kept(A, kept, count, lens, lost, pages, columns):
    seqs, cache = _filled(A, pages=pages, rows=1, columns=columns, lens=_ints(10))
    seqs.room(12)
    from w4a16_linear_amd.attention_module import token_slots
    slots = token_slots(seqs.page_table, 10 + torch.arange(12, dtype=torch.int32, device=DEV)[None], 16, pages)[0]
    cache.k_scale.view(-1)[slots[slots >= 0].long()] = 5000.0 + torch.arange(12, device=DEV)[slots >= 0]
    seqs.accept([cache], _ints(*kept)[None], _ints(count))
    assert seqs.lens.tolist() == [lens] and seqs.lost.tolist() == [lost]
    assert _held(seqs, cache, 0) == [1000.0 + i for i in range(10)] + [5000.0 + i for i in kept[:lens - 10]]
    seqs.room(0)
    seqs.room(1)
    assert seqs.lens.tolist() == [lens] and seqs.lost.tolist() == [lost]


def test_steps_in_a_graph(A):
    """accept, fork and room captured: replays on new contents equal eager steps."""
    start, cache = _filled(A, pages=6, rows=3, columns=3, lens=_ints(20, 9, 0))
    other = A.new_cache(6, 1, 16, 64, "fp8")
    held = [start.page_table.clone(), start.lens.clone(), _ints(0, 2, -1, 0, -1, -1, -1, -1, -1).view(3, 3), _ints(2, 1, 0),
            _ints(0, 0, 1)]
    scale = cache.k_scale.clone()

    def step(c, table, lens, kept, count, parents):
        from w4a16_linear_amd.attention_module import PagedSequences
        seqs = PagedSequences(3, 3, 6, 16)
        seqs.page_table, seqs.lens = table, lens
        seqs.room(4)
        seqs.accept([c], kept, count)
        first = seqs.page_table, seqs.lens, seqs.lost
        seqs.fork([c], parents)
        seqs.room(1)
        return (*first, seqs.page_table, seqs.lens, seqs.lost, seqs.missing)

    step(cache, *held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(cache, *held)
    for i, parents in enumerate(([0, 0, 1], [0, 0, 0], [1, 0, 1], [-1, 2, 1])):
        held[4].copy_(torch.tensor(parents, dtype=torch.int32))
        held[3].copy_(torch.tensor([2, i % 2, 0], dtype=torch.int32))
        held[2][1, 0] = i % 2 - 1
        cache.k_scale.copy_(scale)
        other.k_scale.copy_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = step(other, *held)
        torch.cuda.synchronize()
        assert all(torch.equal(r, w) for r, w in zip(res, want)) and torch.equal(cache.k_scale, other.k_scale)


@pytest.mark.parametrize("pages,columns", [(9, 4), (14, 3), (40, 6)])
def test_rows_always_hold_their_tokens(A, pages, columns):
    """Random steps in pools that run out at times: drafted, accepted, forked, dropped, compacted.  After
    each, every row holds the tokens that a plain list of them says, and `lost` counts the others."""
    import numpy as np
    from w4a16_linear_amd.attention_module import PagedSequences, token_slots
    rng = np.random.default_rng(pages)
    rows, page, draft = 5, 16, 9
    seqs, cache = PagedSequences(rows, columns, pages, page), A.new_cache(pages, 1, page, 64, "fp8")
    tokens, lost, mark, short = [[] for _ in range(rows)], [0] * rows, 0, 0

    def compare():
        assert seqs.lens.tolist() == [len(t) for t in tokens] and seqs.lost.tolist() == lost
        for row, want in enumerate(tokens):
            assert _held(seqs, cache, row) == want

    for step in range(60):
        kind = rng.random()
        if kind < 0.6:
            short += int(seqs.room(draft)) > 0
            places = seqs.lens[:, None] + torch.arange(draft, dtype=torch.int32, device=DEV)
            slots = token_slots(seqs.page_table, places, page, pages)
            marks = mark + torch.arange(rows * draft, device=DEV).view(rows, draft).float()
            mark += rows * draft
            cache.k_scale.view(-1)[slots[slots >= 0].long()] = marks[slots >= 0]
            kept, count = np.full((rows, draft), -1, np.int32), rng.integers(0, draft + 1, rows).astype(np.int32)
            for b in range(rows):
                kept[b, :count[b]] = np.sort(rng.permutation(draft)[:count[b]])
                has = slots[b].tolist()
                stored = [float(marks[b, i]) for i in kept[b, :count[b]] if has[i] >= 0]
                tokens[b] = tokens[b] + stored
                lost[b] += int(count[b]) - len(stored)
            seqs.accept([cache], torch.from_numpy(kept).to(DEV), torch.from_numpy(count).to(DEV))
        elif kind < 0.9:
            parents = rng.integers(-1, rows + 1, rows)
            missing = int(seqs.fork([cache], torch.from_numpy(parents.astype(np.int32)).to(DEV)))
            short += missing > 0
            ended = seqs.lens.tolist()
            old, new = [(tokens[a], lost[a]) if 0 <= a < rows else ([], 0) for a in parents], []
            for (t, c), n in zip(old, ended):
                assert n == len(t) or n == len(t) // page * page
                missing -= n != len(t)
                new.append((t[:n], c + len(t) - n))
            assert missing == 0
            tokens, lost = [t for t, _ in new], [c for _, c in new]
        else:
            seqs.compact([cache])
        compare()
    assert (short > 0) == (pages < rows * columns)


def test_a_refused_call_leaves_the_rows(A):
    """A cache that cannot be copied in is refused before the table changes."""
    seqs, cache = _filled(A, pages=8, rows=3, columns=3, lens=_ints(20, 9, 0))
    before = [seqs.page_table, seqs.lens, seqs.lost]
    host = A.new_cache(8, 1, 16, 64, "fp8", device="cpu")
    for call in (lambda: seqs.fork([cache, host], _ints(0, 0, 1)), lambda: seqs.compact([cache, host]),
                 lambda: seqs.fork([cache], _ints(0, 0, 1).long())):
        with pytest.raises(ValueError):
            call()
        assert seqs.page_table is before[0] and seqs.lens is before[1] and seqs.lost is before[2]
        for row, n in enumerate((20, 9, 0)):
            assert _held(seqs, cache, row) == [1000.0 * (row + 1) + i for i in range(n)]
