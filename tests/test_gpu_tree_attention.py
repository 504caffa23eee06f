"""Attention of drafted tokens over the paged cache against the float64 oracle, for every
cache format, head width and number of row tiles; masks that leave rows empty, sequences
without a token, pages in any order, tokens that hold NaN behind a mask."""
import math

import numpy as np
import pytest
import torch

from oracle import attention_oracle as AO
from w4a16_linear_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32, UBF = 2.0 ** -24, 2.0 ** -8   # half an ulp of 1 in float32 and bfloat16


def _garbage(cache, rng):
    """Fill every row of a cache with what an uninitialised buffer may hold: any code
    bits (also NaN patterns) and any scale."""
    for t in (cache.k, cache.v, cache.k_sign, cache.v_sign):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.from_numpy(rng.integers(0, 256, tuple(b.shape), dtype=np.uint8)))
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))


class Problem:
    """A filled cache with sequences of the given lengths (cached tokens, then `draft` drafted)."""

    def __init__(self, seed, fmt, dim, heads, kv_heads, lens, draft, page=16, spare=3, alpha=0.73, q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.draft, self.heads, self.kv = rng, lens, draft, heads, kv_heads
        batch = len(lens)
        per = max(1, -(-(max(lens) + draft) // page)) + 1
        pages = batch * per + spare
        self.cache = A.new_cache(pages, kv_heads, page, dim, fmt, alpha, DEV)
        _garbage(self.cache, rng)
        ids = rng.permutation(pages)[:batch * per].reshape(batch, per).astype(np.int32)
        self.keys, self.values = [], []
        for b, n in enumerate(lens):
            t = n + draft
            x = [torch.from_numpy(rng.standard_normal((t, kv_heads, dim)).astype(np.float32)).to(DEV)
                 for _ in range(2)]
            slots = ids[b, np.arange(t) // page] * page + np.arange(t) % page
            A.cache_write(self.cache, x[0], x[1], torch.from_numpy(slots.astype(np.int32)).to(DEV))
            k, v = A.cache_read(self.cache, torch.from_numpy(slots.astype(np.int32)).to(DEV), torch.float32)
            self.keys.append(k.double().cpu().numpy())
            self.values.append(v.double().cpu().numpy())
            ids[b, max(1, -(-t // page)):] = rng.choice([-1, 2 ** 31 - 1, pages])   # never read
        self.slots_of = lambda b, at: int(ids[b, at // page]) * page + at % page
        self.table = torch.from_numpy(ids).to(DEV)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        fused = torch.from_numpy((q_gain * rng.standard_normal((batch, draft, (heads + 2) * dim))).astype(np.float32))
        self.q = fused.to(DEV, torch.bfloat16)[..., dim:(heads + 1) * dim].unflatten(-1, (heads, dim))

    def check(self, out, lse, seen, counts=None, scale=None):
        """seen [batch, draft, draft]; holds every output to its error bound."""
        dim, share = self.cache.dim, self.heads // self.kv
        scale = dim ** -0.5 if scale is None else scale
        q = self.q.double().cpu().numpy()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, n in enumerate(self.lens):
            c = self.draft if counts is None else counts[b]
            ok = np.array(seen[b]).copy()
            ok[:, c:] = False
            for h in range(self.kv):
                of = slice(h * share, (h + 1) * share)
                ref, rl, spread, reach = AO.attention(q[b][:, of], self.keys[b][:, h], self.values[b][:, h],
                                                      n, ok, scale)
                ref[c:], rl[c:], spread[c:], reach[c:] = 0.0, -np.inf, 0.0, 0.0
                got, gl = out[b][:, of], lse[b][:, of]
                assert np.array_equal(np.isneginf(rl), np.isneginf(gl))
                # a score: dim products summed in float32, two scalings, the exponential's ulps
                # (its argument is a difference of two scores); the sum over the keys in float32
                keys = n + self.draft
                e_s = (dim + 8) * 2 * U32 * reach
                e_l = (keys / 16 + 80) * U32
                fin = np.isfinite(rl)
                assert (np.abs(gl - rl)[fin] <= (2 * e_s + e_l + 4 * U32 * (np.abs(rl) + 1))[fin]).all()
                # weights rounded to bfloat16, the result rounded to bfloat16
                rel = UBF * 1.01 + 4 * e_s + 2 * e_l + 8 * U32
                bound = rel[..., None] * spread + UBF * 1.01 * np.abs(ref) + 1e-38
                err = np.abs(got - ref)
                assert (err <= bound).all(), (b, h, float((err / (bound + 1e-300)).max()))


def _words(seen):
    seen = np.asarray(seen)
    draft = seen.shape[-1]
    w = np.zeros(seen.shape[:-1] + (-(-draft // 32),), np.uint32)
    for j in range(draft):
        w[..., j // 32] |= seen[..., j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32)).to(DEV)


def _chain(batch, draft):
    return np.broadcast_to(np.tril(np.ones((draft, draft), bool)), (batch, draft, draft))


LENS = [0, 1, 15, 16, 17, 31, 33, 130, 257]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv,draft", [(4, 2, 1), (3, 3, 5), (8, 1, 4), (14, 2, 9), (5, 1, 33)])
def test_against_oracle(gpu_lib, fmt, dim, heads, kv, draft):
    """One row tile to several workgroups of rows; random masks, some rows wholly empty."""
    p = Problem(dim + heads + draft, fmt, dim, heads, kv, LENS, draft)
    seen = p.rng.random((len(LENS), draft, draft)) < 0.5
    seen[:, 0] = False
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, _words(seen), return_lse=True)
    p.check(out, lse, seen)
    assert not out[0, 0].any() and torch.isneginf(lse[0, 0]).all()      # nothing seen at all
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    p.check(out, lse, _chain(len(LENS), draft))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_split_over_workgroups(gpu_lib, fmt, page):
    """Long sequences in pieces, short ones in the same batch with one piece or none; a
    shared tree; an upper bound of the lengths that is too low."""
    lens, draft = [3000, 0, 70, 1999], 6
    p = Problem(page, fmt, 128, 8, 2, lens, draft, page=page)
    parents = torch.tensor([[-1, 0, 0, 1, -1, 4]], dtype=torch.int32)
    words = A.tree_mask(parents)[0].contiguous().to(DEV)
    bits = words.cpu().numpy().view(np.uint32)[:, 0]
    seen = np.broadcast_to((bits[:, None] >> np.arange(draft)) & 1, (4, draft, draft)).astype(bool)
    assert A.attention_workspace_bytes(4, draft, 8, 2, 128, 3000) > 0
    first = None
    for max_len in (3000, 500, 0, None):
        out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, words, max_len=max_len, return_lse=True)
        p.check(out, lse, seen)
        if max_len == 3000:
            first = (out, lse)
    for _ in range(3):      # the same call gives the same bits
        out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, words, max_len=3000, return_lse=True)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("draft", [1, 20])
def test_values_near_the_largest(gpu_lib, fmt, draft):
    """Powers of two pass through: values 2^118 times as large give exactly that much larger
    results (no weight exceeds 1, so hundreds of keys leave the sums within float32)."""
    n, dim, page = 500, 64, 16
    k, v = (torch.randn(n + draft, 2, dim, device=DEV).clamp(-3, 3) for _ in range(2))
    k = k * 0.1
    q = torch.randn(1, draft, 4, dim, device=DEV).bfloat16()
    ids = torch.arange(-(-(n + draft) // page), dtype=torch.int32, device=DEV)
    slots = torch.arange(n + draft, dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out = []
    for grow in (1.0, 2.0 ** 118):
        cache = A.new_cache(len(ids), 2, page, dim, fmt, device=DEV)
        A.cache_write(cache, k, v * grow, slots)
        out.append(A.tree_attention(q, cache, ids[None], lens).float())
    assert torch.isfinite(out[1]).all() and torch.equal(out[0] * 2.0 ** 118, out[1])


@pytest.mark.parametrize("fmt", ["fp8", "opq4"])
@pytest.mark.parametrize("dim,draft", [(64, 1), (128, 1), (256, 1), (128, 9)])
def test_many_pieces(gpu_lib, fmt, dim, draft):
    """A sequence in more pieces than a wave joins at once, beside one with fewer."""
    lens = [12001, 4097]
    p = Problem(dim + draft, fmt, dim, 6, 1, lens, draft, page=64)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    p.check(out, lse, _chain(2, draft))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_counts(gpu_lib, fmt):
    lens, draft, counts = [5, 40, 0, 2000, 9], 7, [0, 3, 2, 7, 1]
    p = Problem(3, fmt, 64, 6, 2, lens, draft)
    ct = torch.tensor(counts, dtype=torch.int32, device=DEV)
    seen = p.rng.random((5, draft, draft)) < 0.6
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, _words(seen), counts=ct, return_lse=True)
    p.check(out, lse, seen, counts)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, counts=ct, return_lse=True)
    p.check(out, lse, _chain(5, draft), counts)
    assert not out[0].any() and not out[1, 3:].any()
    # outside 0..draft: clamped
    wild = torch.tensor([-5, 100, 2 ** 31 - 1, 7, -2 ** 31], dtype=torch.int32, device=DEV)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, counts=wild, return_lse=True)
    p.check(out, lse, _chain(5, draft), [0, 7, 7, 7, 0])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_behind_a_mask_stays_there(gpu_lib, fmt, bad):
    """A drafted token with NaN keys and values: rows that see it are NaN, the others do not
    notice it."""
    lens, draft = [20, 300], 4
    p = Problem(9, fmt, 128, 4, 2, lens, draft)
    x = torch.randn(1, 2, 128, device=DEV)
    x[0, 0, 7] = bad                      # kv head 0 only
    for b, n in enumerate(lens):
        slot = torch.tensor([p.slots_of(b, n + 2)], dtype=torch.int32, device=DEV)
        A.cache_write(p.cache, x, x, slot)
        k, v = A.cache_read(p.cache, slot, torch.float32)
        for h in range(2):
            p.keys[b][n + 2, h], p.values[b][n + 2, h] = k[0, h].cpu().numpy(), v[0, h].cpu().numpy()
    seen = np.ones((2, draft, draft), bool)
    seen[:, [0, 3], 2] = False            # rows 0 and 3 do not see token 2
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, _words(seen), return_lse=True)
    assert torch.isnan(out[:, 1:3, :2]).all() and torch.isnan(lse[:, 1:3, :2]).all()
    assert torch.isfinite(out[:, [0, 3]]).all() and torch.isfinite(out[:, :, 2:]).all()
    clean = [k.copy() for k in p.keys], [v.copy() for v in p.values]
    for b, n in enumerate(lens):          # what rows 1 and 2 of head 0 give is not compared
        p.keys[b][n + 2, 0] = p.values[b][n + 2, 0] = 0.0
    q = p.q.clone()
    keep = torch.tensor([0, 3], device=DEV)
    sub = out[:, keep], lse[:, keep]
    p.q, p.draft = q, draft
    full_out, full_lse = out.clone(), lse.clone()
    ref = seen.copy()
    ref[:, 1:3] = seen[:, 1:3]
    full_out[:, 1:3, :2], full_lse[:, 1:3, :2] = 0.0, -math.inf
    for b in range(2):
        for h in range(2):
            of = slice(2 * h, 2 * h + 2)
            r, rl, spread, _ = AO.attention(q[b, :, of].double().cpu().numpy(), p.keys[b][:, h], p.values[b][:, h],
                                            lens[b], seen[b], 128 ** -0.5)
            rows = [0, 3] if h == 0 else [0, 1, 2, 3]
            err = np.abs(full_out[b, rows, of].double().cpu().numpy() - r[rows])
            assert (err <= 2 * UBF * spread[rows] + 2 * UBF * np.abs(r[rows])).all()
            assert np.allclose(full_lse[b, rows, of].double().cpu().numpy(), rl[rows], rtol=0, atol=1e-5)
    assert len(clean) == 2 and sub[0].shape[1] == 2


def test_nan_query_stays_in_its_row(gpu_lib):
    p = Problem(12, "fp8", 128, 8, 2, [100], 3)
    q = p.q.clone()
    ref, _ = A.tree_attention(q, p.cache, p.table, p.lens_t, return_lse=True)
    q[0, 1, 5, 3] = float("nan")
    out, lse = A.tree_attention(q, p.cache, p.table, p.lens_t, return_lse=True)
    assert torch.isnan(out[0, 1, 5]).all() and torch.isnan(lse[0, 1, 5])
    out[0, 1, 5] = ref[0, 1, 5]
    assert torch.equal(out, ref)


@pytest.mark.parametrize("gain", [0.0, 1e-3, 30.0, 300.0])
def test_flat_and_peaked_scores(gpu_lib, gain):
    """From equal weights to one token taking all: the running maximum moves often."""
    p = Problem(21, "fp8", 64, 4, 1, [500, 3], 2, q_gain=gain)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    p.check(out, lse, _chain(2, 2))
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, scale=-0.5, return_lse=True)
    p.check(out, lse, _chain(2, 2), scale=-0.5)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_rising_scores(gpu_lib, fmt):
    """Scores that rise along the sequence: every step raises the maximum."""
    p = Problem(22, fmt, 64, 2, 1, [700], 1)
    base = torch.randn(64, device=DEV)
    for at in range(701):
        p.keys[0][at, 0] = (base * (at / 100.0)).cpu().numpy()
    x = torch.from_numpy(p.keys[0]).float().to(DEV)
    v = torch.from_numpy(p.values[0]).float().to(DEV)
    slots = torch.tensor([p.slots_of(0, a) for a in range(701)], dtype=torch.int32, device=DEV)
    A.cache_write(p.cache, x, v, slots)
    k, v = A.cache_read(p.cache, slots, torch.float32)
    p.keys, p.values = [k.double().cpu().numpy()], [v.double().cpu().numpy()]
    p.q = base.bfloat16().expand(1, 1, 2, 64).contiguous()
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    p.check(out, lse, _chain(1, 1))


def test_page_outside_the_cache_is_nan(gpu_lib):
    p = Problem(30, "opq4", 64, 2, 1, [40, 40], 1)
    p.table[0, 1] = p.cache.pages
    p.table[1, 2] = -7
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_lengths_beyond_the_page_table_are_clamped(gpu_lib):
    p = Problem(31, "fp8", 64, 2, 1, [15], 1)     # 16 tokens fill page 0; page 1 is never read
    table = p.table[:, :1].contiguous()
    ref = A.tree_attention(p.q, p.cache, table, p.lens_t)
    for wild in (16, 17, 2 ** 31 - 1):           # no room for the drafted token: the page's 16 tokens
        out = A.tree_attention(p.q, p.cache, table, torch.full_like(p.lens_t, wild))
        assert torch.equal(out, ref)
    out, lse = A.tree_attention(p.q, p.cache, table, torch.full_like(p.lens_t, -3), counts=torch.zeros_like(p.lens_t),
                                return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    none = torch.zeros((1, 0), dtype=torch.int32, device=DEV)
    out, lse = A.tree_attention(p.q, p.cache, none, p.lens_t, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_long_cache_past_32_bits(gpu_lib, fmt):
    """Rows whose byte offsets pass 2^32: the last pages of a large cache."""
    dim, heads, page = 256, 8, 256
    row = {"bf16": 512, "fp8": 256, "opq4": 128}[fmt]
    pages = (5 << 30) // (row * heads * page)
    cache = A.new_cache(pages, heads, page, dim, fmt, device=DEV)
    tokens = 300
    ids = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device=DEV)
    at = torch.arange(tokens, device=DEV)
    slots = (ids[0][at // page] * page + at % page).to(torch.int32)
    k, v = (torch.randn(tokens, heads, dim, device=DEV) for _ in range(2))
    A.cache_write(cache, k, v, slots)
    gk, gv = A.cache_read(cache, slots, torch.float32)
    assert (gk - k).norm() < 0.1 * k.norm()
    q = torch.randn(1, 1, heads, dim, device=DEV).bfloat16()
    out = A.tree_attention(q, cache, ids, torch.tensor([tokens - 1], dtype=torch.int32, device=DEV))
    s = torch.einsum("hd,thd->ht", q[0, 0].double().cpu(), gk.double().cpu()) / 16.0
    ref = torch.einsum("ht,thd->hd", torch.softmax(s, -1), gv.double().cpu())
    assert (out[0, 0].double().cpu() - ref).abs().max() < 0.02
    del cache


def test_index_arrays_that_start_inside_others(gpu_lib):
    """A part of a batch, its arrays sliced: the rows of the whole batch's result."""
    lens, draft = [70, 33, 200], 5
    p = Problem(77, "fp8", 64, 4, 2, lens, draft)
    seen = p.rng.random((3, draft, draft)) < 0.5
    words, counts = _words(seen), torch.tensor([5, 3, 4], dtype=torch.int32, device=DEV)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, words, counts, return_lse=True)
    p.check(out, lse, seen, counts.tolist())
    for b in (1, 2):
        part, part_lse = A.tree_attention(p.q[b:], p.cache, p.table[b:], p.lens_t[b:], words[b:], counts[b:],
                                          return_lse=True)
        assert torch.equal(part, out[b:]) and torch.equal(part_lse, lse[b:])


def test_another_stream_and_graph(gpu_lib):
    """Captured once and replayed with eager work between: every replay equals the eager call,
    and follows lengths changed in place."""
    p = Problem(40, "opq4", 128, 8, 2, [2500, 900], 3)
    lens = p.lens_t.clone()
    ref, ref_lse = A.tree_attention(p.q, p.cache, p.table, lens, max_len=2500, return_lse=True)
    shorter = torch.tensor([2300, 17], dtype=torch.int32, device=DEV)
    ref2, _ = A.tree_attention(p.q, p.cache, p.table, shorter, max_len=2500, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = A.tree_attention(p.q, p.cache, p.table, lens, max_len=2500)
    s.synchronize()
    assert torch.equal(out, ref)
    buf = torch.empty_like(ref)
    ws = torch.empty(A.attention_workspace_bytes(2, 3, 8, 2, 128, 2500), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        A.tree_attention(p.q, p.cache, p.table, lens, max_len=2500, out=buf, workspace=ws)
    for i in range(4):
        buf.zero_()
        lens.copy_(shorter if i % 2 else p.lens_t)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, ref2 if i % 2 else ref)
        A.tree_attention(p.q, p.cache, p.table, lens, max_len=2500)
    assert torch.isfinite(ref_lse).all()


def test_refusals_and_empty(gpu_lib):
    p = Problem(50, "fp8", 64, 4, 2, [20], 2)
    args = dict(q=p.q, cache=p.cache, page_table=p.table, lens=p.lens_t)
    assert A.tree_attention(p.q[:, :0], p.cache, p.table, p.lens_t).shape == (1, 0, 4, 64)
    w = torch.zeros((1, 2, 1), dtype=torch.int32, device=DEV)
    for bad in (dict(q=p.q.float()), dict(q=p.q[..., :32]), dict(q=p.q[:, :, :3]), dict(lens=p.lens_t.long()),
                dict(page_table=p.table[0]), dict(mask=w[:, :1]), dict(mask=w.long()), dict(counts=p.lens_t.float()),
                dict(max_len=10 ** 6), dict(scale=float("nan")), dict(out=torch.empty_like(p.q).float()),
                dict(q=p.q.transpose(2, 3))):
        with pytest.raises(ValueError):
            A.tree_attention(**{**args, **bad})


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("draft", [1, 20])
@pytest.mark.parametrize("power", [20, 27, 33, 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores(gpu_lib, fmt, draft, power, sign):
    """Scores around +-2^power, so far apart that one key takes all: its value comes out,
    with its score as the log-sum, however coarse float32 is there.  Keys w_j p, queries
    +-2^power p / dim for a pattern p of signs: the products and their sum are exact but for
    the stored w_j."""
    lens, dim, heads, kv = [0, 1, 300, 5000], 64, 4, 2
    p = Problem(power + draft, fmt, dim, heads, kv, lens, draft, page=64)
    pattern = p.rng.choice([-1.0, 1.0], dim)
    for b, n in enumerate(lens):
        step = np.concatenate([p.rng.integers(70, 117, n), 10 + p.rng.permutation(draft)])
        if n > 1:
            step[p.rng.permutation(n)[:2]] = 1, 124           # the prefix's only least and only largest
        keys = (0.5 + step[:, None] / 256.0) * pattern
        x = torch.from_numpy(np.repeat(keys[:, None], kv, 1).astype(np.float32)).to(DEV)
        slots = torch.tensor([p.slots_of(b, a) for a in range(n + draft)], dtype=torch.int32, device=DEV)
        A.cache_write(p.cache, x, torch.from_numpy(p.values[b]).float().to(DEV), slots)
        k, v = A.cache_read(p.cache, slots, torch.float32)
        p.keys[b], p.values[b] = k.double().cpu().numpy(), v.double().cpu().numpy()
    q = torch.from_numpy(sign * 2.0 ** power / dim * pattern).to(DEV, torch.bfloat16).expand(4, draft, heads, dim)
    out, lse = A.tree_attention(q.contiguous(), p.cache, p.table, p.lens_t, scale=1.0, return_lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        for t in range(draft):
            for h in range(heads):
                s = p.keys[b][:n + t + 1, h // 2] @ (sign * 2.0 ** power / dim * pattern)
                best = int(s.argmax())
                assert len(s) == 1 or s[best] - np.partition(s, -2)[-2] > 100.0
                v = p.values[b][best, h // 2]
                # the weight rounded to bfloat16, the result rounded to bfloat16
                assert (np.abs(out[b, t, h] - v) <= 2.02 * UBF * np.abs(v)).all(), (b, t, h)
                # dim products summed in float32, two scalings, the factor ln 2
                assert abs(lse[b, t, h] - s[best]) <= (dim + 16) * 2 * U32 * abs(s[best]), (b, t, h)


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim,draft", [(64, 1), (64, 16), (128, 1), (128, 5), (256, 1), (256, 40)])
@pytest.mark.parametrize("gain", [1.0, 0.05])
def test_weights_at_twice_their_bits(gpu_lib, fmt, dim, draft, gain):
    """With one tile of rows, and for wide heads, on bf16 and fp8 caches the weights go in with
    twice bfloat16's bits.  Each sequence has two tokens with values that nearly cancel, so
    that a result is small beside its parts and its own rounding hides nothing; the drafted
    tokens see only those two.  With small queries, whose scores' worst case is small too,
    weights rounded to bfloat16 would break the bound nearly everywhere."""
    batch, heads = 16, 2
    p = Problem(dim + draft, fmt, dim, heads, heads, [2] * batch, draft, q_gain=gain)
    q = p.q.double().cpu().numpy()
    scale = dim ** -0.5
    for b in range(batch):
        k = p.keys[b]
        s = scale * np.einsum("hd,thd->th", q[b, 0], k[:2])
        v = p.values[b].copy()
        v[1] = -np.exp(s[0] - s[1])[:, None] * v[0]              # cancels for the first drafted token
        slots = torch.tensor([p.slots_of(b, a) for a in range(2 + draft)], dtype=torch.int32, device=DEV)
        # the keys as they were: codes of their own values (each row's largest is a code's value)
        A.cache_write(p.cache, torch.from_numpy(k).float().to(DEV), torch.from_numpy(v).float().to(DEV), slots)
        k, v = A.cache_read(p.cache, slots, torch.float32)
        p.keys[b], p.values[b] = k.double().cpu().numpy(), v.double().cpu().numpy()
    seen = np.zeros((batch, draft, draft), bool)
    out = A.tree_attention(p.q, p.cache, p.table, p.lens_t, _words(seen)).double().cpu().numpy()
    broken = 0
    for b in range(batch):
        for h in range(heads):
            ref, _, spread, reach = AO.attention(q[b][:, h:h + 1], p.keys[b][:, h], p.values[b][:, h], 2, seen[b], scale)
            # a score's errors as in Problem.check, in every weight and in their sum of two;
            # each weight in two parts of 8 bits (2^-17), float32 products and sums; the result
            e_s = (dim + 8) * 2 * U32 * reach
            rel = 2.0 ** -17 * 1.01 + 4 * e_s + 16 * U32
            bound = rel[..., None] * spread + UBF * 1.01 * np.abs(ref) + 1e-38
            assert (np.abs(out[b][:, h:h + 1] - ref) <= bound).all(), (b, h)
            # the planted mistake, on the CPU: the weights rounded to bfloat16 once
            s = scale * q[b][0, h] @ p.keys[b][:2, h].T
            w = np.exp(s - s.max())
            once = _bf16(w) @ p.values[b][:2, h] / w.sum()
            broken += int((np.abs(once - ref[0, 0]) > bound[0, 0]).any())
    assert gain == 1.0 or broken >= batch * heads // 2


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 8, 2, 32), (128, 8, 1, 64), (256, 4, 2, 16)])
def test_prompt(gpu_lib, fmt, dim, heads, kv, page):
    """A prompt as one chain of 333 tokens: many groups of rows, each with its own end of the
    keys, alone and after tokens that are cached already."""
    lens, draft = [0, 77], 333
    p = Problem(dim + page, fmt, dim, heads, kv, lens, draft, page=page)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, return_lse=True)
    p.check(out, lse, _chain(2, draft))
    counts = [333, 200]
    ct = torch.tensor(counts, dtype=torch.int32, device=DEV)
    out, lse = A.tree_attention(p.q, p.cache, p.table, p.lens_t, counts=ct, return_lse=True)
    p.check(out, lse, _chain(2, draft), counts)
