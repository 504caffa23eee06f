"""The oracle of pages and drafts tied to facts other than itself: tables worked out by hand, and
the law of what verification lets through, added up exactly over all random numbers."""
import itertools
from fractions import Fraction

import numpy as np
import pytest

from oracle import serving_oracle as SO


def test_resize_by_hand():
    table = [[5, 2, -1, -1], [0, 9, 3, 1], [-1, -1, -1, -1]]
    # row 0 needs three pages and lacks one, row 1 gives up two, row 2 takes one; page 9 is no page
    out, missing = SO.resize(table, [33, 17, 1], 8, 16)
    assert out.tolist() == [[5, 2, 1, -1], [0, 3, -1, -1], [4, -1, -1, -1]] and missing == 0
    out, missing = SO.resize([[0, -1], [-1, -1]], [32, 32], 2, 16)
    assert out.tolist() == [[0, 1], [-1, -1]] and missing == 2
    out, missing = SO.resize([[0, 1]], [-5], 2, 16)
    assert out.tolist() == [[-1, -1]] and missing == 0


def test_fork_by_hand():
    table = [[4, 6, -1], [4, 5, 2]]
    # row 0 twice: its last page (6, half full) stays with the first; row 1 dropped; an empty row
    out, lens, src, dst, missing = SO.fork(table, [24, 40], [0, 7, 0], 8, 16)
    assert out.tolist() == [[4, 6, -1], [-1, -1, -1], [4, 0, -1]] and lens.tolist() == [24, 0, 24]
    assert src.tolist() == [-1, -1, 6] and dst.tolist() == [-1, -1, 0] and missing == 0
    # a row cut back into a page that another holds in full gets a copy, though it is the first
    out, lens, src, dst, missing = SO.fork([[4, 6, 7], [4, 6, -1]], [48, 20], [1, 0], 8, 16)
    assert out.tolist() == [[4, 0, -1], [4, 6, 7]] and src.tolist() == [6, -1] and dst.tolist() == [0, -1]
    # full rows share everything; no page is left for a third end
    out, lens, src, dst, missing = SO.fork([[0, 1]], [32], [0, 0], 2, 16)
    assert out.tolist() == [[0, 1], [0, 1]] and src.tolist() == [-1, -1] and missing == 0
    out, lens, src, dst, missing = SO.fork([[0, 1]], [17], [0, 0], 2, 16)
    assert out.tolist() == [[0, 1], [0, -1]] and missing == 1


def test_compact_by_hand():
    out, src, dst, used = SO.compact([[7, 1, -1], [7, 4, 12]], 8)
    assert used == 3 and src == [4, 7] and dst == [0, 2]
    assert out.tolist() == [[2, 1, -1], [2, 0, -1]]


# Probabilities in eighths; random numbers run over the cells their borders cut [0, 1) into.

def _law(p, tokens, q=None, parents=None, cells=64):
    """Exact law of the token after node 0 (kept child's token, or next), every random number over
    the middles of `cells` equal cells that no border cuts."""
    draft, vocab = len(tokens), len(p[0])
    law = [Fraction(0)] * vocab
    for us in itertools.product(range(cells), repeat=draft):
        u = [(c + 0.5) / cells for c in us]
        kept, number, nxt, _ = SO.verify(p, tokens, u, q, parents)
        law[tokens[kept[1]] if number > 1 else nxt] += Fraction(1, cells ** draft)
    return law


def test_a_draft_models_chain_keeps_the_targets_law():
    p = [[4 / 8, 1 / 8, 3 / 8], [1 / 8, 1 / 8, 6 / 8]]
    q = [[2 / 8, 4 / 8, 2 / 8]]
    law = [Fraction(0)] * 3
    for x in range(3):
        for v, f in enumerate(_law(p, [0, x], q, cells=48)):
            law[v] += f * Fraction(q[0][x])
    # u q < p is decided at p / q (1/4 for the second token), the residual at 2/3
    assert law == [Fraction(4, 8), Fraction(1, 8), Fraction(3, 8)]


@pytest.mark.parametrize("tokens,parents,cells", [([0, 1], [-1, 0], 56), ([0, 0, 2], [-1, 0, 0], 16),
                                                  ([0, 2, 2], [-1, 0, 0], 40)])
def test_candidates_keep_the_targets_law(tokens, parents, cells):
    p = [[4 / 8, 1 / 8, 3 / 8]] * 3
    law = _law(p, tokens, None, parents, cells)
    assert law == [Fraction(4, 8), Fraction(1, 8), Fraction(3, 8)]


def test_verify_by_hand():
    p = [[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]
    assert SO.verify(p, [9, 1, 1], [0.0, 0.2, 0.9])[:3] == ([0, 1, 2], 3, 0)
    assert SO.verify(p, [9, 1, 1], [0.5, 0.25, 0.0])[:3] == ([0, -1, -1], 1, 0)       # 0.25 is not below 0.25
    assert SO.verify(p, [9, 1, 0], [0.99, 0.2, 0.0])[:3] == ([0, 1, -1], 2, 1)        # p = 0 is never kept
    assert SO.verify(p, [9, 7, 0], [0.6, 0.0, 0.0])[:3] == ([0, -1, -1], 1, 1)        # no such token
    assert SO.verify(p, [9, 1, 1], [0.0, 0.2, 0.9], count=2)[:3] == ([0, 1, -1], 2, 1)
    assert SO.verify(p, [9, 1, 1], [0.0, 0.2, 0.9], count=0)[:3] == ([-1, -1, -1], 0, -1)
    q = [[0.0, 0.75, 0.25], [0.0, 1.0, 0.0]]
    assert SO.verify(p, [9, 1, 1], [0.9, 0.5, 0.5], q)[:3] == ([0, -1, -1], 1, 0)     # 0.375 >= 0.25; p - q leaves 0
    assert SO.verify([[0.0, 0.0]], [0], [0.5])[:3] == ([0], 1, -1)


@pytest.mark.parametrize("plant", ["owner", "freed_first", "z", "next_from_p", "strict"])
def test_planted_mistakes_show(plant, monkeypatch):
    """Each plausible mistake changes an answer that is worked out above."""
    if plant == "owner":       # the last row keeps the page instead of the first
        a = SO.fork([[4, 6, -1]], [24], [0, 0], 8, 16)
        assert a[0].tolist() == [[4, 6, -1], [4, 0, -1]]
    elif plant == "freed_first":  # a dropped row's pages are free for this very call
        monkeypatch.setattr(SO, "_free", lambda named, pages: [p for p in range(pages) if p not in named and p not in (0, 1)])
        assert SO.fork([[0, 1, -1], [4, 6, -1]], [20, 20], [1, 1], 8, 16)[3].tolist() != [-1, 0]
    elif plant == "z":         # siblings after the first need a smaller number
        p = [[0.5, 0.25, 0.25]] * 3
        assert SO.verify(p, [0, 0, 1], [0.0, 0.7, 0.45], None, [-1, 0, 0])[0] == [0, 2, -1]
        assert SO.verify(p, [0, 0, 1], [0.0, 0.7, 0.55], None, [-1, 0, 0])[0] == [0, -1, -1]
    elif plant == "next_from_p":
        p, q = [[0.5, 0.5]] * 2, [[1.0, 0.0]]
        assert SO.verify(p, [0, 0], [0.0, 0.9], q)[2] == 1
    else:
        monkeypatch.setattr(SO, "draw", lambda w, u: next(i for i in range(len(w)) if sum(w[:i + 1]) >= u * sum(w)))
        assert SO.draw([0.0, 0.5, 0.5], 0.0) != 1
