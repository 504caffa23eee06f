"""Calls at the stated maxima and past 2^31 elements: what lies far out is computed as what lies near."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from test_gpu_adapters import DEV, U32, _gen, _stack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu_lib):
    from w4a16_linear_amd import adapters
    adapters.load()
    return adapters


@pytest.fixture(scope="module")
def A(gpu_lib):
    from w4a16_linear_amd import attention
    attention.load()
    return attention


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _sample(m, g):
    return torch.cat((torch.randint(0, m, (1000,), generator=g, device=DEV), torch.arange(m - 200, m, device=DEV)))


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


@pytest.mark.parametrize("m,k,n", [(1 << 22, 8, 8), ((1 << 19) + 3, 32, 4104)])   # the most tokens; m n past 2^31
def test_adapters(L, m, k, n):
    g = _gen(m)
    a = _stack(L, 3, 8, k, n, g)
    x, y = _normal((m, k), g), _normal((m, n), g)
    index = torch.randint(-1, 3, (m,), generator=g, device=DEV, dtype=torch.int32)
    at = _sample(m, g)
    got = L.lowrank_add(y, x, a, index)
    # few elements a row, so that the sums over k are taken in one piece in any call: bit for bit
    assert torch.equal(got[at], L.lowrank_add(y[at], x[at], a, index[at]))
    del got
    dx, down, up = L.lowrank_backward(y, x, a, index, dx_dtype=torch.float32)
    e = torch.zeros((at.numel(), 8), dtype=torch.float64, device=DEV)
    for i in range(3):
        some = index[at] == i
        e[some] = a.scale[i].double() * (y[at][some].double() @ a.up[i].double().T)
        size = a.scale[i].double() * (y[at][some].double().abs() @ a.up[i].double().abs().T) @ a.down[i].double().abs()
        want = e[some] @ a.down[i].double()
        assert ((dx[at][some].double() - want).abs() <= (n + 200) * U32 * size).all()
    assert not dx[at][index[at] < 0].any()
    want, size = ([torch.zeros(t.shape, dtype=torch.float64, device=DEV) for t in (a.down, a.up)] for _ in range(2))
    for t in range(0, m, 1 << 18):
        for i in range(3):
            some = t + torch.nonzero(index[t:t + (1 << 18)] == i)[:, 0]
            xs, ys, s = x[some].double(), y[some].double(), a.scale[i].double()
            for to, f in ((want, lambda v: v), (size, torch.abs)):
                to[0][i] += (s * f(ys) @ f(a.up[i].double()).T).T @ f(xs)
                to[1][i] += (s * f(xs) @ f(a.down[i].double()).T).T @ f(ys)
    for r, w, b in zip((down, up), want, size):
        # sums of up to m / 128 products a wave and of as many slots, below 2^-24 times their number of the terms
        assert ((r.double() - w).abs() <= (n + m // 32 + 500) * U32 * b).all()
        assert ((r.double() - w).abs().max() <= 1e-4 * w.abs().max())


def test_linear_backward_of_many_tokens(L, gpu_lib):
    g = _gen(1)
    m, n, k = (1 << 20) + 5, 2104, 32                       # dy and its padded copy past 2^31
    w = gpu_lib.quantize(torch.randn((n, k), generator=g, device=DEV), 0.73)
    dy = _normal((m, n), g)
    got = L.linear_backward(dy, w, 0.73, out_dtype=torch.float32)
    at, full = _sample(m, g), gpu_lib.dequantize(w, 0.73).double()
    want, size = dy[at].double() @ full, dy[at].double().abs() @ full.abs()
    assert ((got[at].double() - want).abs() <= (n + 64) * U32 * size).all()


@pytest.mark.parametrize("m", [8, 100, 520])
def test_linear_backward_of_a_large_weight(L, gpu_lib, m):
    g = _gen(m)
    n = k = 65536
    w = gpu_lib.QuantizedWeight(torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=g, device=DEV, dtype=torch.int32),
                                torch.randint(-2 ** 31, 2 ** 31, (n, k // 32), generator=g, device=DEV, dtype=torch.int32),
                                torch.rand(n, generator=g, device=DEV))
    dy = _normal((m, n), g)
    got = L.linear_backward(dy, w, 0.73, out_dtype=torch.float32)
    full = gpu_lib.dequantize(w, 0.73)
    at = torch.cat((torch.randint(0, k, (100,), generator=g, device=DEV), torch.arange(k - 64, k, device=DEV)))
    some = full[:, at].double()
    want, size = dy.double() @ some, dy.double().abs() @ some.abs()
    assert ((got[:, at].double() - want).abs() <= (n + 64) * U32 * size).all()
    assert ((got[:, at].double() - want).abs().max() <= 1e-4 * want.abs().max())


def test_verify(A):
    g = _gen(3)
    draft, vocab = 520, 1 << 22                             # the largest vocabulary; the last rows past 2^31
    p = torch.rand((1, draft, vocab), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    t = torch.randint(0, vocab, (1, draft), generator=g, device=DEV, dtype=torch.int32)
    p[0, torch.arange(draft - 1, device=DEV), t[0, 1:].long()] = 0.5
    u = torch.full((1, draft), 0.25, device=DEV)
    u[0, 518], u[0, 0] = 0.75, 0.999999                     # 517 are kept, the next is not

    class Rows:
        def __getitem__(self, i):
            return p[0, i].float().cpu().numpy()

    kept, count, following = A.verify_drafts(p, t, u)
    want = SO.verify(Rows(), t[0].tolist(), u[0].tolist())
    assert kept[0].tolist() == want[0] and int(count) == want[1] == 518 and int(following) == want[2] > vocab // 2


def test_pages(A):
    rng = np.random.default_rng(0)
    rows, columns, pages, page = 1 << 20, 2, 1 << 20, 16    # the most of both
    table = np.full((rows, columns), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    held = rng.permutation(rows)[:rows // 4]
    ids = rng.permutation(pages)[:rows // 2].reshape(-1, 2)
    table[held] = ids
    lens[held] = rng.integers(1, 2 * page + 1, held.size)
    dev = [torch.from_numpy(v).to(DEV) for v in (table, lens)]
    more = np.where(rng.random(rows) < 0.9, lens + rng.integers(0, 2 * page, rows), lens).astype(np.int32)
    got = A.pages_resize(dev[0], torch.from_numpy(more).to(DEV), pages, page)
    want = SO.resize(table, more, pages, page)              # more than there are
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and int(got[1]) == want[1] > 0
    parents = rng.integers(-1, rows, rows).astype(np.int32)
    got = A.pages_fork(dev[0], dev[1], torch.from_numpy(parents).to(DEV), pages, page)
    want = SO.fork(table, lens, parents.tolist(), pages, page)
    for r, w in zip(got, want):
        assert np.array_equal(r.cpu().numpy().squeeze(), np.squeeze(w))
    got = A.pages_compact(dev[0], pages)
    used = np.unique(table[table >= 0])
    src, dst = used[used >= used.size], np.setdiff1d(np.arange(used.size), used)
    to = np.arange(pages + 1)                               # the last is for no page
    to[src], to[pages] = dst, -1
    n = src.size
    assert np.array_equal(got[0].cpu().numpy(), to[table]) and int(got[3]) == used.size
    assert np.array_equal(got[1][:n].cpu().numpy(), src) and np.array_equal(got[2][:n].cpu().numpy(), dst)
    assert (got[1][n:] == -1).all() and (got[2][n:] == -1).all()


def test_copies_of_far_pages(A):
    g = _gen(4)
    cache = A.new_cache(1 << 20, 2, 16, 128, "fp8")         # 4 GB of codes a side
    codes = cache.k.view(torch.uint8)
    codes.random_(0, 100, generator=g)
    ids = torch.randperm(1 << 20, generator=g, device=DEV)[:4000].to(torch.int32)
    src, dst = ids[:2000].clone(), ids[2000:].clone()
    if not (dst == (1 << 20) - 1).any() and not (src == (1 << 20) - 1).any():
        dst[0] = (1 << 20) - 1
    want = codes[src.long()]
    before = codes[5000:6000].clone()
    A.cache_copy_pages(cache, src, dst)
    assert torch.equal(codes[dst.long()], want) and torch.equal(codes[src.long()], want)
    other = torch.ones(1000, dtype=torch.bool, device=DEV)
    near = dst[(dst >= 5000) & (dst < 6000)].long() - 5000
    other[near] = False
    assert torch.equal(codes[5000:6000][other], before[other])
