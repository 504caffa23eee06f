"""Pages of a cache on the GPU against the plain oracle: every number equal."""
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _pool(rng, rows, columns, pages, page, beams=4, wild=0.0):
    """A table whose groups of rows share their first pages, and lengths."""
    table, lens = np.full((rows, columns), -1, np.int64), np.zeros(rows, np.int64)
    ids = rng.permutation(pages)
    at = 0
    for i in range(rows):
        held = int(rng.integers(0, columns + 1))
        if i % beams == 0:
            prompt = ids[at:at + held // 2]
            at += len(prompt)
        share = min(len(prompt), held)
        table[i, :share] = prompt[:share]
        own = ids[at:at + held - share]
        at += len(own)
        held = share + len(own)
        table[i, share:held] = own
        lens[i] = max(0, held * page - int(rng.integers(0, page)))
        if rng.random() < 0.3:
            lens[i] = lens[i] // page * page                # no page partly filled
    if wild:
        hit = rng.random(table.shape) < wild
        table[hit] = rng.choice([-1, -7, pages, 2 ** 31 - 1, -2 ** 31], hit.sum())
    return table, lens


# rows, columns, pages, page: the last ones are past what one workgroup takes
SIZES = [(1, 1, 1, 16), (3, 5, 40, 16), (16, 7, 33, 32), (40, 65, 700, 16), (31, 300, 16384, 64), (7, 64, 2048, 128),
         (64, 600, 9000, 16), (1500, 33, 16000, 16), (12, 20, 16385, 64), (1030, 70, 70001, 16)]


@pytest.mark.parametrize("rows,columns,pages,page", SIZES)
@pytest.mark.parametrize("wild", [0.0, 0.1])
def test_resize(A, rows, columns, pages, page, wild):
    rng = np.random.default_rng(rows + columns)
    table, lens = _pool(rng, rows, columns, pages, page, wild=wild)
    want = lens + rng.integers(-3 * page, 3 * page, rows)
    if wild:
        want[rng.random(rows) < 0.1] = 2 ** 31 - 1
        want[rng.random(rows) < 0.1] = -2 ** 31
    out, missing = A.pages_resize(_dev(table), _dev(want), pages, page)
    ref, ref_missing = SO.resize(table, want, pages, page)
    assert np.array_equal(out.cpu().numpy(), ref) and missing.tolist() == [ref_missing]
    t = _dev(table)
    same, _ = A.pages_resize(t, _dev(want), pages, page, out=t)
    assert same is t and torch.equal(t, out)


@pytest.mark.parametrize("rows,columns,pages,page", SIZES)
@pytest.mark.parametrize("wild", [0.0, 0.1])
def test_fork(A, rows, columns, pages, page, wild):
    rng = np.random.default_rng(rows * 3 + columns)
    table, lens = _pool(rng, rows, columns, pages, page, wild=wild)
    if wild:                                                # rows cut back into shared pages, odd lengths
        cut = rng.random(rows) < 0.3
        lens[cut] = lens[cut] // 2
        lens[rng.random(rows) < 0.1] = 2 ** 31 - 1
        lens[rng.random(rows) < 0.1] = -5
    for made in (rows, max(1, rows // 2), 2 * rows + 1):
        parents = rng.integers(-1 if wild else 0, rows + (1 if wild else 0), made)
        got = A.pages_fork(_dev(table), _dev(lens), _dev(parents), pages, page)
        ref = SO.fork(table, lens, parents, pages, page)
        for g, r in zip(got[:4], ref[:4]):
            assert np.array_equal(g.cpu().numpy(), r)
        assert got[4].tolist() == [ref[4]]


@pytest.mark.parametrize("rows,columns,pages,page", SIZES)
@pytest.mark.parametrize("wild", [0.0, 0.1])
def test_compact(A, rows, columns, pages, page, wild):
    rng = np.random.default_rng(rows * 5 + columns)
    table, _ = _pool(rng, rows, columns, pages, page, wild=wild)
    ref, src, dst, used = SO.compact(table, pages)
    out, s, d, u = A.pages_compact(_dev(table), pages)
    room = min(pages // 2, rows * columns)
    assert np.array_equal(out.cpu().numpy(), ref) and u.tolist() == [used]
    assert s.tolist() == src + [-1] * (room - len(src)) and d.tolist() == dst + [-1] * (room - len(dst))
    t = _dev(table)
    assert A.pages_compact(t, pages, out=t)[0] is t and torch.equal(t, out)


def test_empty(A):
    none = torch.empty((0, 5), dtype=torch.int32, device=DEV)
    no = torch.empty(0, dtype=torch.int32, device=DEV)
    table, missing = A.pages_resize(none, no, 9, 16)
    assert table.shape == (0, 5) and missing.tolist() == [0]
    out = A.pages_fork(none, no, _dev([0, -1]), 9, 16)
    assert out[0].tolist() == [[-1] * 5] * 2 and out[1].tolist() == [0, 0] and out[4].tolist() == [0]
    assert A.pages_fork(_dev([[3]]), _dev([5]), no, 9, 16)[0].shape == (0, 1)
    table, src, dst, used = A.pages_compact(none, 9)
    assert src.numel() == 0 and used.tolist() == [0]
    flat = torch.empty((4, 0), dtype=torch.int32, device=DEV)
    assert A.pages_resize(flat, _dev([1, 2, 3, 4]), 9, 16)[1].tolist() == [0]
    assert A.pages_fork(flat, _dev([1, 2, 3, 4]), _dev([1]), 9, 16)[1].tolist() == [0]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("heads,page,dim", [(1, 16, 64), (3, 32, 128), (8, 64, 128), (5, 16, 256)])
def test_copy_pages(A, fmt, heads, page, dim):
    g = torch.Generator(device=DEV)
    g.manual_seed(heads + dim)
    pages = 37
    cache = A.new_cache(pages, heads, page, dim, fmt)
    slots = torch.arange(pages * page, dtype=torch.int32, device=DEV)
    kv = [torch.randn((pages * page, heads, dim), generator=g, device=DEV) for _ in range(2)]
    A.cache_write(cache, kv[0], kv[1], slots)
    before = [None if t is None else t.clone() for t in (cache.k, cache.k_sign, cache.k_scale, cache.v, cache.v_sign, cache.v_scale)]
    src = [3, 5, -1, 9, 36, 7, 11, 2, 40]
    dst = [4, 6, 8, -1, 0, 7, 37, -2 ** 31, 10]
    A.cache_copy_pages(cache, _dev(src), _dev(dst))
    after = (cache.k, cache.k_sign, cache.k_scale, cache.v, cache.v_sign, cache.v_scale)
    for old, new in zip(before, after):
        if old is None:
            continue
        for a, b in ((3, 4), (5, 6), (36, 0)):
            old.view(torch.uint8)[b] = old.view(torch.uint8)[a]
        assert torch.equal(old.view(torch.uint8), new.view(torch.uint8))


def test_a_pool_in_use(A):
    """Requests come, grow, fork and go; after every step each row reads its own tokens back."""
    rng = np.random.default_rng(1)
    pages, page, heads, dim, rows, columns = 96, 16, 2, 64, 8, 12
    cache = A.new_cache(pages, heads, page, dim, "bf16")
    table = torch.full((rows, columns), -1, dtype=torch.int32, device=DEV)
    held = [[] for _ in range(rows)]                         # what each row's tokens were written as
    lens = np.zeros(rows, np.int64)
    stamp = 0

    def read_back():
        slots, want = [], []
        t = table.cpu().numpy()
        for i in range(rows):
            for j, v in enumerate(held[i]):
                slots.append(int(t[i, j // page]) * page + j % page)
                want.append(v)
        if slots:
            k, v = A.cache_read(cache, _dev(slots), out_dtype=torch.float32)
            w = torch.tensor(want, dtype=torch.float32, device=DEV)[:, None, None]
            assert torch.equal(k, w.expand_as(k)) and torch.equal(v, -w.expand_as(v))

    for step in range(40):
        add = rng.integers(0, 12, rows)
        add = np.minimum(add, columns * page - lens)
        table, missing = A.pages_resize(table, _dev(lens + add), pages, page)
        assert missing.tolist() == [0]
        t, slots, values = table.cpu().numpy(), [], []
        for i in range(rows):
            for j in range(int(lens[i]), int(lens[i] + add[i])):
                stamp = (stamp + 1) % 256
                held[i].append(float(stamp))
                slots.append(int(t[i, j // page]) * page + j % page)
                values.append(float(stamp))
        lens = lens + add
        if slots:
            kv = torch.tensor(values, device=DEV)[:, None, None].expand(-1, heads, dim).contiguous()
            A.cache_write(cache, kv, -kv, _dev(slots))
        read_back()
        parents = rng.integers(0, rows, rows)
        parents[rng.random(rows) < 0.3] = -1
        table, new_lens, src, dst, missing = A.pages_fork(table, _dev(lens), _dev(parents), pages, page)
        assert missing.tolist() == [0]
        A.cache_copy_pages(cache, src, dst)
        held = [list(held[a]) if a >= 0 else [] for a in parents]
        lens = new_lens.cpu().numpy().astype(np.int64)
        assert lens.tolist() == [len(h) for h in held]
        read_back()
        if step % 5 == 4:
            table, src, dst, used = A.pages_compact(table, pages)
            A.cache_copy_pages(cache, src, dst)
            assert int(table.max()) < int(used)
            read_back()


def test_refusals(A):
    t, lens = _dev(np.zeros((4, 6))), _dev(np.zeros(4))
    buf = torch.zeros(100, dtype=torch.int32, device=DEV)
    for call in (lambda: A.pages_resize(t, lens[:3], 9, 16), lambda: A.pages_resize(t.long(), lens, 9, 16),
                 lambda: A.pages_resize(t.t(), lens, 9, 16), lambda: A.pages_resize(t, lens, 9, 24),
                 lambda: A.pages_resize(t, lens, 0, 16), lambda: A.pages_resize(t, lens, 2 ** 20 + 1, 16),
                 lambda: A.pages_resize(buf[:24].view(4, 6), lens, 9, 16, out=buf[6:30].view(4, 6)),
                 lambda: A.pages_resize(t, lens, 9, 16, workspace=buf[:8]),
                 lambda: A.pages_fork(t, lens, lens, 9, 16, out=t), lambda: A.pages_fork(t, lens, lens.cpu(), 9, 16),
                 lambda: A.pages_compact(buf[:24].view(4, 6), 9, out=buf[4:28].view(4, 6)),
                 lambda: A.pages_compact(t[0], 9)):
        with pytest.raises(ValueError):
            call()
    cache = A.new_cache(4, 1, 16, 64, "fp8")
    with pytest.raises(ValueError):
        A.cache_copy_pages(cache, lens, lens[:2])
    with pytest.raises(ValueError):
        A.cache_copy_pages(cache, t, t)


@pytest.mark.parametrize("rows,columns,pages", [(96, 5, 700), (97, 5, 700), (64, 256, 16384), (65, 256, 16384), (8, 9, 16384),
                                                (8, 9, 16385), (200, 60, 16000), (300, 60, 16000)])
def test_at_the_change_of_paths(A, rows, columns, pages):
    for wild in (0.0, 0.1):
        test_resize(A, rows, columns, pages, 16, wild)
        test_fork(A, rows, columns, pages, 16, wild)
        test_compact(A, rows, columns, pages, 16, wild)
