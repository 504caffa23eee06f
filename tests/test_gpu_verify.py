"""Verification of drafted tokens on the GPU against the plain float64 oracle: every number equal."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def A(gpu_lib):
    from w4a16_linear_amd import attention
    attention.load()
    return attention


def _case(seed, batch, draft, vocab, kind, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    logits = torch.randn((batch, draft, vocab), generator=g, device=DEV) * 2.5
    p = torch.softmax(logits, -1).to(dtype)
    u = torch.rand((batch, draft), generator=g, device=DEV)
    q = parents = None
    if kind == "drawn":
        q = torch.softmax(logits[:, :draft - 1] + 0.7 * torch.randn((batch, draft - 1, vocab), generator=g, device=DEV), -1)
        q = q.to(dtype)
        t = torch.zeros((batch, draft), dtype=torch.long, device=DEV)
        if draft > 1:
            t[:, 1:] = torch.multinomial(q.float().flatten(0, 1), 1, generator=g).view(batch, draft - 1)
    else:
        likely = torch.topk(p.float(), min(vocab, 6), -1).indices
        par = np.tile(np.arange(-1, draft - 1), (batch, 1))
        if kind == "tree":
            for i in range(1, draft):
                par[:, i] = rng.integers(max(0, i - 5), i, batch)
            parents = torch.from_numpy(par.astype(np.int32)).to(DEV)
        pick = torch.from_numpy(rng.integers(0, min(vocab, 6), (batch, draft))).to(DEV)
        node = torch.from_numpy(np.maximum(par, 0)).to(DEV)
        t = likely[torch.arange(batch, device=DEV)[:, None], node, pick]
    return p, t.to(torch.int32), u, q, parents


def _check(got, p, t, u, q, parents, counts=None):
    kept, number, nxt = (g.cpu().numpy() for g in got)
    f = [None if x is None else x.float().cpu().numpy() for x in (p, u, q)]
    t = t.cpu().numpy()
    par = None if parents is None else parents.cpu().numpy()
    for b in range(t.shape[0]):
        want = SO.verify(f[0][b], t[b], f[1][b], None if q is None else f[2][b], None if par is None else par[b].tolist(),
                         None if counts is None else int(counts[b]))
        assert kept[b].tolist() == want[0] and int(number[b]) == want[1], (b, kept[b], want[0])
        assert int(nxt[b]) == want[2], (b, int(nxt[b]), want[2])


@pytest.mark.parametrize("batch,draft,vocab", [(1, 1, 1), (1, 2, 5), (3, 6, 1000), (5, 9, 1025), (2, 33, 4099), (4, 64, 257),
                                               (2, 70, 777), (1, 200, 64), (2, 5, 32003), (130, 4, 16411)])
@pytest.mark.parametrize("kind", ["drawn", "chain", "tree"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify(A, batch, draft, vocab, kind, dtype):
    p, t, u, q, parents = _case(batch + draft + vocab, batch, draft, vocab, kind, dtype)
    got = A.verify_drafts(p, t, u, draft_probs=q, parents=parents)
    if batch > 8:                                            # the oracle takes a while
        pick = torch.arange(0, batch, 17, device=DEV)
        sub = [None if x is None else x[pick] for x in (p, t, u, q, parents)]
        _check([g[pick] for g in got], *sub)
        again = A.verify_drafts(*(x.contiguous() for x in sub[:3]), draft_probs=sub[3], parents=sub[4])
        for a, b in zip(again, got):
            assert torch.equal(a, b[pick])
    else:
        _check(got, p, t, u, q, parents)


@pytest.mark.parametrize("kind", ["drawn", "chain", "tree"])
def test_counts_and_strides(A, kind):
    p, t, u, q, parents = _case(7, 6, 12, 1501, kind, torch.float32)
    counts = torch.tensor([0, 1, 2, 12, 40, -3], dtype=torch.int32, device=DEV)
    wide = torch.full((6, 14, 1601), float("nan"), device=DEV)
    wide[:, 1:13, 37:1538] = p
    view = wide[:, 1:13, 37:1538]
    _check(A.verify_drafts(view, t, u, draft_probs=q, parents=parents, counts=counts), p, t, u, q, parents, counts.tolist())
    one = p[:1].expand(6, -1, -1)                            # every sequence the same probabilities
    _check(A.verify_drafts(one, t, u, draft_probs=q, parents=parents), one, t, u, q, parents)


def test_borders(A):
    """Probabilities in 1/1024 and random numbers on their borders: everything is exact."""
    rng = np.random.default_rng(3)
    batch, draft, vocab = 64, 5, 300
    p = np.zeros((batch, draft, vocab), np.float32)
    for row in p.reshape(-1, vocab):
        cuts = np.sort(rng.integers(0, 1025, 39))
        row[rng.permutation(vocab)[:40]] = np.diff(np.concatenate(([0], cuts, [1024]))) / 1024.0
    u = (rng.integers(0, 1024, (batch, draft)) / 1024.0).astype(np.float32)
    u[:8, 0] = 0.0
    t = np.zeros((batch, draft), np.int32)
    for b in range(batch):
        for i in range(1, draft):
            t[b, i] = rng.choice(np.nonzero(p[b, i - 1])[0])
            if b % 2:
                u[b, i] = p[b, i - 1, t[b, i]]              # not below: refused
    dev = [torch.from_numpy(x).to(DEV) for x in (p, t, u)]
    _check(A.verify_drafts(*dev), *dev, None, None)
    q = np.roll(p, 1, axis=2)[:, :-1].copy()
    dq = torch.from_numpy(q).to(DEV)
    _check(A.verify_drafts(*dev, draft_probs=dq), *dev, dq, None)


def test_values_that_are_no_probabilities(A):
    p = torch.full((4, 2, 2050), 2.0 ** -12, device=DEV)
    p[0, 0, ::3] = float("nan")
    p[0, 1, ::2] = float("inf")
    p[1] = 0.0
    p[2, 0] = -1.0
    p[2, 0, 2049] = 1e-30
    p[3, :, :2049] = 0.0
    t = torch.tensor([[0, 3], [0, 1], [0, -1], [0, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    u = torch.tensor([[0.5, 0.0], [0.5, 0.0], [0.999, 0.0], [0.25, 0.0]], device=DEV)
    _check(A.verify_drafts(p, t, u), p, t, u, None, None)
    _check(A.verify_drafts(p, t, u, draft_probs=p[:, 1:].contiguous()), p, t, u, p[:, 1:], None)
    kept, number, nxt = A.verify_drafts(p, t, u)
    assert number.tolist() == [1, 1, 1, 1] and nxt.tolist()[1:] == [-1, 2049, 2049]


def test_odd_trees(A):
    p, t, u, _, _ = _case(5, 4, 90, 400, "tree", torch.float32)
    rng = np.random.default_rng(5)
    par = rng.integers(-3, 92, (4, 90)).astype(np.int32)     # later, outside, own: never kept
    par[1] = 0                                               # one node, every token under it
    t[1, 1:] = t[1, 1]                                       # all the same token
    par[2] = 0
    parents = torch.from_numpy(par).to(DEV)
    u = u * 0.3
    _check(A.verify_drafts(p, t, u, parents=parents), p, t, u, None, parents)


def test_law_of_what_comes_out(A):
    """Frequencies over many sequences against the target's probabilities."""
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    batch, vocab = 40000, 12
    p = torch.softmax(torch.randn((1, 2, vocab), generator=g, device=DEV), -1)
    q = torch.softmax(torch.randn((1, 1, vocab), generator=g, device=DEV), -1)
    t = torch.zeros((batch, 2), dtype=torch.int32, device=DEV)
    t[:, 1] = torch.multinomial(q[0, 0].expand(batch, -1).contiguous(), 1, generator=g)[:, 0].to(torch.int32)
    u = torch.rand((batch, 2), generator=g, device=DEV)
    for kw in (dict(draft_probs=q.expand(batch, -1, -1)), {}):
        kept, number, nxt = A.verify_drafts(p.expand(batch, -1, -1), t, u, **kw)
        first = torch.where(number > 1, t[:, 1], nxt)
        if kw:                                               # candidates here are drawn too: the law is theirs mixed
            freq = torch.bincount(first, minlength=vocab).double() / batch
            # each frequency within 5 standard deviations
            sd = (p[0, 0].double() * (1 - p[0, 0].double()) / batch).sqrt()
            assert ((freq - p[0, 0].double()).abs() <= 5 * sd).all()
        for x in range(vocab):                               # given the drafted token, chance keeps it with p
            at = t[:, 1] == x
            if not kw and at.sum() > 500:
                px = float(p[0, 0, x])
                assert abs(float((number[at] > 1).double().mean()) - px) <= 5 * (px * (1 - px) / int(at.sum())) ** 0.5


def test_refusals(A):
    p, t, u, q, parents = _case(1, 3, 4, 50, "tree", torch.float32)
    q = p[:, 1:].contiguous()
    for call in (lambda: A.verify_drafts(p.half(), t, u), lambda: A.verify_drafts(p.transpose(1, 2), t, u),
                 lambda: A.verify_drafts(p, t.long(), u), lambda: A.verify_drafts(p, t[:, :3], u),
                 lambda: A.verify_drafts(p, t, u.double()), lambda: A.verify_drafts(p, t, u, draft_probs=q, parents=parents),
                 lambda: A.verify_drafts(p, t, u, draft_probs=q.bfloat16()), lambda: A.verify_drafts(p, t, u, draft_probs=p),
                 lambda: A.verify_drafts(p, t, u, parents=parents[0]), lambda: A.verify_drafts(p, t, u, counts=t[:, 0].long()),
                 lambda: A.verify_drafts(p, t, u, workspace=u[:1]), lambda: A.verify_drafts(p.cpu(), t, u),
                 lambda: A.verify_drafts(p[:, :0], t[:, :0].contiguous(), u[:, :0].contiguous()),
                 lambda: A.verify_drafts(p.expand(3, 4, 50)[:, :1].expand(3, 1025, 50),
                                         t[:, :1].expand(3, 1025).contiguous(), u[:, :1].expand(3, 1025).contiguous())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):
        A.verify_drafts(p.requires_grad_(), t, u)


def _sequence(p, t, u, parents):
    one = [torch.tensor(x, device=DEV)[None] for x in (p, t, u, parents)]
    return one[0].float(), one[1].to(torch.int32), one[2].float(), one[3].to(torch.int32)


def test_a_token_before_its_parent_is_nobodys_sibling(A):
    """Entries under a node that do not come after it were never tested: a later token equal to one
    of them is tested as any other."""
    p = [[0.0, 0.0, 1.0, 0.0], [0.25] * 4, [0.0, 0.8, 0.0, 0.2], [0.25] * 4, [0.25] * 4]
    s = _sequence(p, [0, 1, 2, 3, 1], [0.5, 0.5, 0.1, 0.9, 0.1], [-1, 2, 0, 2, 2])
    assert SO.verify(p, [0, 1, 2, 3, 1], [0.5, 0.5, 0.1, 0.9, 0.1], None, [-1, 2, 0, 2, 2])[0] == [0, 2, 4, -1, -1]
    _check(A.verify_drafts(*s[:3], parents=s[3]), *s[:3], None, s[3])
    even = [[1 / 16] * 16] * 5
    s = _sequence(even, [0, 7, 3, 9, 7], [0.5, 0.5, 0.01, 0.9, 0.01], [-1, 2, 0, 2, 2])
    _check(A.verify_drafts(*s[:3], parents=s[3]), *s[:3], None, s[3])
    # a node's children in its own 64 tokens and in the next ones, equal to a token before the
    # node (not tested) and to one after it (tested)
    for second in (7, 9):
        parents, t = [-1] * 130, [5] * 130
        parents[3], t[3] = 20, 7
        parents[20], t[20] = 0, 1
        parents[40], t[40] = 20, 9
        parents[100], t[100] = 20, second
        parents[129], t[129] = 20, 2
        u = [0.5] + [0.9] * 129
        u[20] = u[100] = 0.01
        s = _sequence([[1 / 16] * 16] * 130, t, u, parents)
        _check(A.verify_drafts(*s[:3], parents=s[3]), *s[:3], None, s[3])


@pytest.mark.parametrize("draft", [5, 63, 130])
def test_trees_with_parents_on_either_side(A, draft):
    rng = np.random.default_rng(draft)
    batch, vocab = 96, 6
    p = torch.from_numpy(rng.dirichlet(np.ones(vocab), (batch, draft)).astype(np.float32)).to(DEV)
    t = torch.from_numpy(rng.integers(0, vocab, (batch, draft)).astype(np.int32)).to(DEV)
    u = np.where(np.arange(draft) % 9 == 0, 0.01, 0.2 + 0.6 * rng.random((batch, draft))).astype(np.float32)
    u = torch.from_numpy(u).to(DEV)
    at = np.arange(draft) // 9 * 9                           # every ninth hangs under the ninth before, the rest beside it
    par = np.where(np.arange(draft) % 9 == 0, at - 9, at + 9 * rng.integers(0, 2, (batch, draft))).astype(np.int32)
    parents = torch.from_numpy(par).to(DEV)
    _check(A.verify_drafts(p, t, u, parents=parents), p, t, u, None, parents)
