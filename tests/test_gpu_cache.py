"""The quantized cache on the GPU against the oracle: codes, signs and scales bit for bit,
values read back, slots that are skipped, rows that hold NaN or nothing."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import attention_oracle as AO
from w4a16_linear_amd import attention as A
from w4a16_linear_amd import workloads as WL

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _stored(cache, side, slots):
    """(code values float64, scale float32) of the rows at slots: [tokens, heads, ...]."""
    codes, sign, scale = (getattr(cache, side), getattr(cache, side + "_sign"), getattr(cache, side + "_scale"))
    page, off = slots // cache.page, slots % cache.page
    scale = scale.cpu().numpy()[page, :, off]
    if cache.fmt == "opq4":
        p, s = WL.u32(codes)[page, :, off], WL.u32(sign)[page, :, off]
        shape = p.shape[:-1]
        q, n = O.unpack(p.reshape(-1, p.shape[-1]), s.reshape(-1, s.shape[-1]))
        v = np.where(n != 0, -1.0, 1.0) * AO.opq_levels(cache.alpha)[q]
        return v.reshape(*shape, -1), scale
    return codes.cpu().double().numpy()[page, :, off], scale


def _expect(x, cache):
    rows = x.float().cpu().numpy().reshape(-1, x.shape[-1])
    c, s = AO.cache_rows(rows, cache.fmt, cache.alpha)
    return c.reshape(x.shape), s.reshape(x.shape[:-1])


def _values(rng, tokens, heads, dim):
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    x *= rng.choice([1.0, 1e-3, 30.0, 2.0 ** -90, 1e30], (tokens, heads, 1)).astype(np.float32)
    x[rng.random(x.shape) < 0.02] *= 8.0
    x[rng.random(x.shape) < 0.02] = 0.0
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt,alpha", [("bf16", 0.73), ("fp8", 0.73), ("opq4", 0.73), ("opq4", 1.0), ("opq4", 3.0),
                                       ("opq4", 0.3)])
def test_rows_bit_for_bit(gpu_lib, fmt, alpha, dim, dtype):
    rng = np.random.default_rng(dim + int(100 * alpha))
    tokens, heads, page, pages = 37, 3, 16, 6
    cache = A.new_cache(pages, heads, page, dim, fmt, alpha, DEV)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    k, v = (torch.from_numpy(_values(rng, tokens, heads, dim)).to(DEV, dtype) for _ in range(2))
    A.cache_write(cache, k, v, torch.from_numpy(slots).to(DEV))
    others = np.setdiff1d(np.arange(pages * page), slots)
    kf, vf = A.cache_read(cache, torch.from_numpy(slots).to(DEV), out_dtype=torch.float32)
    kb, vb = A.cache_read(cache, torch.from_numpy(slots).to(DEV))
    for side, x, f32, bf in (("k", k, kf, kb), ("v", v, vf, vb)):
        codes, scale = _stored(cache, side, slots)
        ref_c, ref_s = _expect(x, cache)
        assert np.array_equal(scale, ref_s)
        assert np.array_equal(codes, ref_c)
        if fmt == "opq4":
            q, n, _ = O.quantize(x.float().cpu().numpy().reshape(-1, dim), alpha)
            p = slots // page
            assert np.array_equal(WL.u32(getattr(cache, side))[p, :, slots % page].reshape(-1, dim // 8), q)
            assert np.array_equal(WL.u32(getattr(cache, side + "_sign"))[p, :, slots % page].reshape(-1, dim // 32), n)
        val = torch.from_numpy(AO.cache_values(ref_c, ref_s))
        assert torch.equal(f32.cpu(), val)            # one rounding of code * scale
        assert torch.equal(bf.cpu(), val.bfloat16())
        assert not _stored(cache, side, others)[1].any()   # nothing else was written


@pytest.mark.parametrize("alpha", [0.05, 0.73, 1.0, 2.5, 60.0])
def test_codes_at_every_decision_point(gpu_lib, alpha):
    """Magnitudes one step to either side of each of the fifteen points, in rows with several
    maxima: where an approximate power would decide wrongly."""
    pts = O.decision_thresholds_f32(alpha).astype(np.float32)
    rows = []
    for m in (1.0, 3.0, 0.7, 1e-20, 7e37, 2.0 ** 127):
        m = np.float32(m)
        with np.errstate(over="ignore", under="ignore"):
            near = (pts * m).astype(np.float32)
        near = near[near < m]
        near = np.concatenate([near, np.nextafter(near, np.float32(0)), np.nextafter(near, m)])
        row = np.zeros(64, np.float32)
        row[:min(63, near.size)] = near[:63]
        row[63] = m
        row[::2] *= -1
        rows.append(row)
    x = torch.from_numpy(np.stack(rows))[:, None].to(DEV)
    cache = A.new_cache(1, 1, 16, 64, "opq4", alpha, DEV)
    A.cache_write(cache, x, x, torch.arange(len(rows), dtype=torch.int32, device=DEV))
    q, n, s = O.quantize(np.stack(rows), alpha)
    assert np.array_equal(WL.u32(cache.k)[0, 0, :len(rows)], q)
    assert np.array_equal(WL.u32(cache.v_sign)[0, 0, :len(rows)], n)
    assert np.array_equal(cache.k_scale.cpu().numpy()[0, 0, :len(rows)], s)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_rows_with_nan_inf_and_nothing(gpu_lib, fmt):
    dim, heads = 128, 2
    x = torch.randn(7, heads, dim)
    x[0, 0, 3] = float("nan")
    x[1, 1, 127] = float("inf")
    x[2, 0, 0] = -float("inf")
    x[3] = 0.0
    x[4] = 2.0 ** -101          # below the smallest row that is kept
    x[5] = 2.0 ** -100
    x[6, 0, 5] = 3.4e38         # overflows bfloat16
    cache = A.new_cache(2, heads, 16, dim, fmt, device=DEV)
    slots = torch.arange(7, dtype=torch.int32, device=DEV)
    A.cache_write(cache, x.to(DEV), x.to(DEV), slots)
    k, v = A.cache_read(cache, slots, out_dtype=torch.float32)
    ref_c, ref_s = _expect(x, cache)
    val = AO.cache_values(ref_c, ref_s)
    for got in (k, v):
        assert np.array_equal(got.cpu().numpy(), val, equal_nan=True)
    assert torch.isnan(k[0, 0]).all() and torch.isfinite(k[0, 1]).all()
    assert torch.isnan(v[1, 1]).all() and torch.isnan(v[2, 0]).all()
    codes, _ = _stored(cache, "k", np.arange(7))
    assert np.isfinite(codes).all()                # no code is ever a NaN


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_skipped_slots(gpu_lib, fmt):
    cache = A.new_cache(2, 1, 16, 64, fmt, device=DEV)
    k = torch.randn(5, 1, 64, device=DEV)
    before = [None if t is None else t.clone() for t in cache[2:]]
    bad = torch.tensor([-1, 32, 2 ** 31 - 1, -2 ** 31, 33], dtype=torch.int32, device=DEV)
    A.cache_write(cache, k, k, bad)
    for a, b in zip(before, cache[2:]):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    A.cache_write(cache, k, k, torch.tensor([31, -1, 0, -1, 16], dtype=torch.int32, device=DEV))
    got, _ = A.cache_read(cache, torch.tensor([31, -1, 0, 32, 16], dtype=torch.int32, device=DEV),
                          out_dtype=torch.float32)
    ref, s = _expect(k, cache)
    val = AO.cache_values(ref, s)
    for i in (0, 2, 4):
        assert np.array_equal(got[i].cpu().numpy(), val[i])
    assert not got[1].any() and not got[3].any()


@pytest.mark.parametrize("fmt", ["fp8", "opq4", "bf16"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (8, 8), (4, 3)])
def test_strided_inputs(gpu_lib, fmt, dtype, offset, pad):
    """Keys and values cut from one fused projection, at any element offset."""
    tokens, heads, dim = 9, 4, 64
    width = 2 * heads * dim + pad
    flat = torch.randn(offset + tokens * width, device=DEV).to(dtype)
    fused = flat[offset:].as_strided((tokens, 2 * heads, dim), (width, dim, 1))
    a, b = (A.new_cache(1, heads, 16, dim, fmt, device=DEV) for _ in range(2))
    slots = torch.arange(tokens, dtype=torch.int32, device=DEV)
    A.cache_write(a, fused[:, :heads], fused[:, heads:], slots)
    A.cache_write(b, fused[:, :heads].contiguous(), fused[:, heads:].contiguous(), slots)
    for s, t in zip(a[2:], b[2:]):
        assert s is None or torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_long_prompt_and_other_stream(gpu_lib):
    """More rows than one wave of workgroups, written and read on a stream of the caller's."""
    tokens, heads, dim, page = 5003, 5, 128, 64
    for fmt in ("fp8", "opq4", "bf16"):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cache = A.new_cache(80, heads, page, dim, fmt, device=DEV)
            k, v = (torch.randn(tokens, heads, dim, device=DEV).bfloat16() for _ in range(2))
            slots = torch.randperm(80 * page, device=DEV)[:tokens].to(torch.int32)
            A.cache_write(cache, k, v, slots)
            gk, gv = A.cache_read(cache, slots)
        s.synchronize()
        pick = torch.arange(0, tokens, 501)
        for x, got in ((k, gk), (v, gv)):
            c, sc = _expect(x[pick.to(DEV)], cache)
            assert torch.equal(got.cpu()[pick], torch.from_numpy(AO.cache_values(c, sc)).bfloat16())
        # every row within half a step of what was written
        step = {"bf16": 0.0, "fp8": 2.0 ** -4, "opq4": 0.06}[fmt]
        top = k.float().abs().amax(-1, keepdim=True)
        off = (gk.float() - k.float()).abs()
        assert (off <= step * (top if fmt == "opq4" else k.float().abs()) + 2.0 ** -9 * top).all()


def test_slots_that_start_inside_an_array(gpu_lib):
    a, b = (A.new_cache(2, 3, 16, 64, "fp8", device=DEV) for _ in range(2))
    x = torch.randn(20, 3, 64, device=DEV)
    slots = torch.randperm(32, device=DEV)[:21].to(torch.int32)
    A.cache_write(a, x, x, slots[1:])
    A.cache_write(b, x, x, slots[1:].clone())
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v_scale, b.v_scale)
    for s, t in zip(A.cache_read(a, slots[3:]), A.cache_read(a, slots[3:].clone())):
        assert torch.equal(s, t)
    A.cache_move(a, slots[None, 1:4], slots[None, 5:8])
    A.cache_move(b, slots[None, 1:4].clone(), slots[None, 5:8].clone())
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v_scale, b.v_scale)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
@pytest.mark.parametrize("dim,tokens", [(64, 9500), (128, 4801), (256, 2402)])
def test_large_calls_equal_small_ones(gpu_lib, fmt, dim, tokens):
    """Enough rows for several heads a group of lanes, with a number of heads that is no
    multiple of theirs: the same bits as tokens written and read a few at a time."""
    heads, page = 7, 32
    k, v = (torch.randn(tokens, heads, dim, device=DEV).bfloat16() for _ in range(2))
    slots = torch.randperm(-(-tokens // page) * page, device=DEV)[:tokens].to(torch.int32)
    slots[100:200] = -1
    a, b = (A.new_cache(-(-tokens // page), heads, page, dim, fmt, device=DEV) for _ in range(2))
    A.cache_write(a, k, v, slots)
    for part in torch.arange(tokens, device=DEV).split(1200):
        A.cache_write(b, k[part], v[part], slots[part])
    for s, t in zip(a[2:], b[2:]):
        assert s is None or torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    for dtype in (torch.bfloat16, torch.float32):
        whole = A.cache_read(a, slots, dtype)
        parts = [A.cache_read(a, slots[part], dtype) for part in torch.arange(tokens, device=DEV).split(1200)]
        for i in range(2):
            assert torch.equal(whole[i], torch.cat([q[i] for q in parts]))
            assert not whole[i][100:200].any()


def test_refusals_and_empty(gpu_lib):
    cache = A.new_cache(2, 2, 16, 64, "fp8", device=DEV)
    k = torch.zeros(3, 2, 64, device=DEV)
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    A.cache_write(cache, k[:0], k[:0], slots[:0])
    assert A.cache_read(cache, slots[:0])[0].shape == (0, 2, 64)
    for args in ((k.half(), k.half(), slots), (k, k.bfloat16(), slots), (k, k[:2], slots), (k, k, slots[:2]),
                 (k, k, slots.long()), (k[:, :1], k[:, :1], slots), (k.transpose(0, 1), k, slots)):
        with pytest.raises(ValueError):
            A.cache_write(cache, *args)
    with pytest.raises(ValueError):
        A.cache_read(cache, slots, out_dtype=torch.float16)
    for bad in (cache._replace(fmt="int8"), cache._replace(k=cache.k.view(torch.uint8)),
                cache._replace(v_scale=cache.v_scale[:1]), cache._replace(fmt="opq4")):
        with pytest.raises(ValueError):
            A.cache_write(bad, k, k, slots)


def test_read_into_shared_memory_is_refused(gpu_lib):
    cache = A.new_cache(2, 2, 16, 64, "fp8", device=DEV)
    slots = torch.arange(5, dtype=torch.int32, device=DEV)
    flat = torch.empty(2 * 5 * 2 * 64 + 64, device=DEV, dtype=torch.bfloat16)
    a, b, c = (flat[i:i + 640].view(5, 2, 64) for i in (0, 640, 576))
    for pair in ((a, a), (a, c), (c, b)):
        with pytest.raises(ValueError, match="share"):
            A.cache_read(cache, slots, out=pair)
    A.cache_read(cache, slots, out=(a, b))
    A.cache_read(cache, slots, out=(b, a))
    A.cache_read(cache, slots[:0], out=(a[:0], a[:0]))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "opq4"])
def test_write_of_several_launches(gpu_lib, fmt):
    """More work-items than one launch's grid counts: of 2^26 tokens all but a few are skipped,
    and those, on both sides of the boundary and at the end, are written as in a small call."""
    dim, tokens, page = 256, 2 ** 26 + 1000, 16
    x = torch.randn(1, 1, dim, device=DEV)
    at = torch.tensor([0, 5, 2 ** 26 - 2, 2 ** 26 - 1, 2 ** 26, 2 ** 26 + 1, tokens - 1], device=DEV)
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    slots[at] = torch.arange(7, dtype=torch.int32, device=DEV) * 3 + 1
    big, small = (A.new_cache(2, 1, page, dim, fmt, device=DEV) for _ in range(2))
    A.cache_write(big, x.expand(tokens, 1, dim), -x.expand(tokens, 1, dim)[:1].expand(tokens, 1, dim), slots)
    A.cache_write(small, x.expand(7, 1, dim).contiguous(), -x.expand(7, 1, dim), slots[at])
    for a, b in zip(big[2:], small[2:]):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert small.k_scale.any()


def test_read_of_several_launches(gpu_lib):
    """2^28 and some rows of 64 read in one call (34 GB a side): the tokens around the boundary
    and the last ones as in a small call, the skipped ones zero."""
    dim, tokens, page = 64, 2 ** 28 + 1000, 16
    cache = A.new_cache(2, 1, page, dim, "fp8", device=DEV)
    A.cache_write(cache, torch.randn(32, 1, dim, device=DEV), torch.randn(32, 1, dim, device=DEV),
                  torch.arange(32, dtype=torch.int32, device=DEV))
    slots = (torch.arange(tokens, dtype=torch.int32, device=DEV) * 7) % 37 - 3
    k, v = A.cache_read(cache, slots)
    for a, b in ((0, 100), (2 ** 28 - 132, 2 ** 28 + 68), (tokens - 100, tokens)):
        for big, small in zip((k, v), A.cache_read(cache, slots[a:b].contiguous())):
            assert torch.equal(big[a:b], small)
    none = slots[-1000:] < 0
    assert not k[-1000:][none].any() and k[-1000:][(slots[-1000:] >= 0) & (slots[-1000:] < 32)].any()
    del k, v
    torch.cuda.empty_cache()
