"""Plain CPU oracle of the attention side: rotary positions, the quantized cache's
rows, and attention of drafted tokens over a cache, in float64 numpy.

TEST INFRASTRUCTURE ONLY.  It shares no code, table or constant generator with the HIP
library; OPQ rows go through the weights' oracle (``quantize``, ``unpack``).
"""
from __future__ import annotations

import math

import numpy as np

from .opq_oracle import alpha_f32, bf16_bits_to_f32, f64_to_bf16_bits, quantize, unpack

SMALLEST = 2.0 ** -100   # quantized rows whose max is below it are stored as zeros


# ------------------------------------------------------------------ rotary

def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_len=0.0,
                       beta_fast=32.0, beta_slow=1.0):
    """(frequencies [rot/2], amplitude)."""
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(base))
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            turns = original_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return np.array(out), (1.0 + 0.1 * math.log(factor) if scaling == "yarn" else 1.0)


def rotary(x, positions, table, layout, sections, backward=False):
    """(result, bound) in float64: x [tokens, heads, dim]; positions [tokens, axes];
    table [len, pairs, 2].  `bound` is the sum of the magnitudes that each
    result adds up (what rounding errors are relative to)."""
    x = np.asarray(x, np.float64)
    table = np.asarray(table, np.float64)
    y, mag = x.copy(), np.abs(x)
    pairs = table.shape[1]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    assert len(axis) == pairs
    for t in range(x.shape[0]):
        for i in range(pairs):
            p = int(positions[t][axis[i]])
            c, s = table[p, i] if 0 <= p < table.shape[0] else (np.nan, np.nan)
            s = -s if backward else s
            a, b = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
            mag[t, :, a] = np.abs(x[t, :, a] * c) + np.abs(x[t, :, b] * s)
            mag[t, :, b] = np.abs(x[t, :, a] * s) + np.abs(x[t, :, b] * c)
    return y, mag


# ------------------------------------------------------------------- cache

def round_e4m3(r):
    """float64 values within +-448 to the nearest e4m3 value, ties to the even one."""
    r = np.asarray(r, np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -20))), -6.0)
    step = 2.0 ** (e - 3)
    return np.rint(r / step) * step


def cache_rows(x32, fmt, alpha=0.73):
    """What rows x32 [n, dim] (float32) are stored as: (values of the codes, scale)
    with the value of an element code * scale; float64 codes, float32 scale."""
    x32 = np.ascontiguousarray(x32, np.float32)
    codes = np.zeros(x32.shape, np.float64)
    scale = np.zeros(x32.shape[0], np.float32)
    for i, row in enumerate(x32):
        if fmt == "bf16":
            with np.errstate(invalid="ignore", over="ignore"):
                v = _bf16_of_f32(row)
            if np.isfinite(v).all():
                codes[i], scale[i] = v, 1.0
            else:
                scale[i] = np.nan
            continue
        if not np.isfinite(row).all():
            scale[i] = np.nan
            continue
        m = np.abs(row).max()
        if float(m) < SMALLEST:
            continue
        if fmt == "fp8":
            s = np.float32(m / np.float32(448.0))
            codes[i] = round_e4m3(np.clip((row / s).astype(np.float32), -448.0, 448.0))
            scale[i] = s
        else:
            packed, sign, sc = quantize(row[None], alpha)
            q, neg = unpack(packed, sign)
            codes[i] = np.where(neg[0] != 0, -1.0, 1.0) * opq_levels(alpha)[q[0]]
            scale[i] = sc[0]
    return codes, scale


def _bf16_of_f32(row):
    b = row.view(np.uint32).astype(np.uint64)
    nan = np.isnan(row)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16) & 0xFFFFFFFF
    out = r.astype(np.uint32).view(np.float32).astype(np.float64)
    out[nan] = np.nan
    return out


def opq_levels(alpha):
    """bfloat16 nearest to (q/15)^(1/alpha), q = 0..15, as float64."""
    g = np.array([(q / 15.0) ** (1.0 / alpha_f32(alpha)) for q in range(16)])
    return bf16_bits_to_f32(f64_to_bf16_bits(g)).astype(np.float64)


def cache_values(codes, scale):
    """float32 values that stored rows stand for (one rounding of code * scale)."""
    with np.errstate(invalid="ignore"):
        return (np.asarray(codes, np.float32) * np.asarray(scale, np.float32)[..., None])


# --------------------------------------------------------------- attention

def attention(q, keys, values, length, seen, scale):
    """One sequence and kv head, all in float64.  q [draft, share, dim]; keys, values
    [tokens, dim] with tokens >= length + draft; seen [draft, draft] booleans.
    Returns out, lse, and for error bounds: the sum of p |v| per output, and the
    largest sum |q| |k| per row."""
    draft, share, dim = q.shape
    out = np.zeros((draft, share, dim))
    lse = np.full((draft, share), -np.inf)
    spread = np.zeros((draft, share, dim))
    reach = np.zeros((draft, share))
    for t in range(draft):
        at = list(range(length)) + [length + j for j in range(draft) if seen[t, j]]
        if not at:
            continue
        k, v = keys[at], values[at]
        for h in range(share):
            s = scale * (k @ q[t, h])
            m = s.max()
            e = np.exp(s - m)
            l = e.sum()
            out[t, h] = (e / l) @ v
            lse[t, h] = m + math.log(l)
            spread[t, h] = (e / l) @ np.abs(v)
            reach[t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, spread, reach
