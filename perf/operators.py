"""The attention-side operators (rotary positions, a quantized paged cache, attention of
drafted tokens over it): the workloads they are measured on, and their plain forms.

`run` computes an operator in elementary torch operations in float32 where `own` is false,
and calls the framework (w4a16_linear_amd.attention) where it is true.  `exact` gives the
same outputs in float64 from the definitions, written apart from the plain forms.

Definitions (w4a16_linear_amd.attention documents them for users):
  rotary   table[p][i] = (cos, sin); a pair (a, b) becomes (a c - b s, a s + b c); the backward
           pass turns the other way.  Pairs are (i, i + rot/2) ("half") or (2i, 2i + 1)
           ("interleaved"); pair i looks the table up at the position of its section's axis.
  cache    one row per (page, head, offset) of `dim` values, with one float32 scale s:
           bf16: values as they are, s = 1;
           fp8:  s = max|x| / 448, codes e4m3(x / s), value code * s;
           opq4: s = max|x|, u = |x| / s in binary32, q = nearest(15 u^alpha) packed eight to a
                 word, a sign plane, value +-bf16((q/15)^(1/alpha)) * s.
  attention  token t of the T drafted ones sees the cached tokens before the draft and the
           drafted tokens that its mask row has a bit for; out = softmax(scale q k) v.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ALPHA = 0.73
CODE_BYTES = {"bf16": 2.0, "fp8": 1.0, "opq4": 0.625}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # queries and keys of eight sequences, one new token each, cut from the fused projection
        dict(name="rotary, one token each", op="rotary", tokens=8, heads=40, row_heads=48, dim=128,
             rot=128, layout="half", axes=1, dtype="bf16", grad=False, table=32768),
        # queries and keys of 4096 image tokens at the framework's hidden size, three position axes
        dict(name="rotary, image tokens", op="rotary", tokens=4096, heads=60, row_heads=90, dim=128,
             rot=128, layout="interleaved", axes=3, dtype="bf16", grad=False, table=1536),
        # a training step's gradient, half of the head turned, odd number of tokens
        dict(name="rotary, gradient", op="rotary", tokens=8191, heads=32, row_heads=32, dim=128,
             rot=64, layout="half", axes=1, dtype="f32", grad=True, table=8192),
        # one decode step of 48 sequences into an 8-bit cache
        dict(name="cache write, one token each", op="write", tokens=48, heads=8, dim=128, page=64,
             fmt="fp8", dtype="bf16"),
        # a long prompt into the framework's own 4-bit codes
        dict(name="cache write, prompt", op="write", tokens=16384, heads=8, dim=128, page=64,
             fmt="opq4", dtype="bf16"),
        # a short shared prefix handed to another attention
        dict(name="cache read, short", op="read", tokens=777, heads=8, dim=64, page=16, fmt="fp8",
             dtype="bf16"),
        # a long history handed to another attention
        dict(name="cache read, long", op="read", tokens=131072, heads=8, dim=128, page=64,
             fmt="opq4", dtype="bf16"),
        # one user, one new token
        dict(name="attention, one sequence", op="attention", batch=1, draft=1, heads=32, kv_heads=8,
             dim=128, page=64, fmt="fp8", longest=1000, ragged=False),
        # a serving batch with sequences of many lengths
        dict(name="attention, batch", op="attention", batch=32, draft=1, heads=32, kv_heads=8,
             dim=128, page=64, fmt="fp8", longest=8191, ragged=True),
        # two very long contexts
        dict(name="attention, long context", op="attention", batch=2, draft=1, heads=64, kv_heads=8,
             dim=128, page=256, fmt="opq4", longest=200000, ragged=False),
        # a tree of drafted tokens to be verified for each of eight sequences
        dict(name="attention, draft trees", op="attention", batch=8, draft=48, heads=32, kv_heads=8,
             dim=128, page=32, fmt="bf16", longest=6001, ragged=True),
        # wide heads, every query head with its own keys, an odd tree, pages smaller than a tile
        dict(name="attention, wide heads", op="attention", batch=3, draft=21, heads=16, kv_heads=16,
             dim=256, page=16, fmt="fp8", longest=4093, ragged=True),
    ]


MOST_BYTES = 420e6     # no more than the largest listed case
MOST_FLOPS = 22e9


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("rotary", "write", "read", "attention", "attention", "attention"))
        if op == "rotary":
            dim = rng.choice((64, 80, 96, 128, 192, 256))
            rot = rng.choice((dim, dim, dim // 2, dim // 4))
            heads = rng.randint(1, 64)
            case = dict(op=op, tokens=_log(rng, 1, 16384), heads=heads,
                        row_heads=heads + rng.choice((0, 0, heads, 5)), dim=dim, rot=rot,
                        layout=rng.choice(("half", "interleaved")),
                        axes=3 if rot % 16 == 0 and rng.random() < 0.3 else 1,
                        dtype=rng.choice(("bf16", "bf16", "f32")), grad=rng.random() < 0.4,
                        table=rng.choice((2048, 8192, 32768)))
        elif op in ("write", "read"):
            case = dict(op=op, tokens=_log(rng, 1, 16384) if op == "write" else _log(rng, 16, 131072),
                        heads=rng.choice((1, 2, 4, 5, 8, 16)), dim=rng.choice((64, 128, 128, 256)),
                        page=rng.choice((16, 32, 64, 128, 256)),
                        fmt=rng.choice(("bf16", "fp8", "fp8", "opq4", "opq4")),
                        dtype=rng.choice(("bf16", "bf16", "f32")))
        else:
            kv_heads = rng.choice((1, 2, 4, 8, 8, 16))
            draft = rng.choice((1, 1, 1, 2, 5, 8, 16, 31, 48, 64))
            case = dict(op=op, batch=_log(rng, 1, 48), draft=draft,
                        heads=kv_heads * rng.choice((1, 2, 3, 4, 4, 7, 8)), kv_heads=kv_heads,
                        dim=rng.choice((64, 128, 128, 256)), page=rng.choice((16, 32, 64, 128, 256)),
                        fmt=rng.choice(("bf16", "fp8", "fp8", "opq4", "opq4")),
                        longest=_log(rng, 1, 200000), ragged=rng.random() < 0.5)
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _lens(case):
    """Cached tokens before the draft, per sequence: `longest` for the first one and, in a
    ragged batch, shares of it spread evenly over (0, 1] in a mixed order."""
    b, longest = case["batch"], case["longest"]
    if not case["ragged"]:
        return [longest] * b
    return [max(0, int(longest * (1.0 - (i * 0.6180339887498949) % 1.0))) for i in range(b)]


def work(case):
    op = case["op"]
    if op == "rotary":
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["heads"]
        rows = min(case["tokens"], case["table"])
        return {"bytes": 2 * n * case["dim"] * es + rows * case["rot"] * 4 + 4 * case["axes"] * case["tokens"],
                "flops": 3 * n * case["rot"]}
    if op in ("write", "read"):
        es = 2 if case["dtype"] == "bf16" else 4
        rows = 2 * case["tokens"] * case["heads"]
        code = rows * (case["dim"] * CODE_BYTES[case["fmt"]] + 4)
        if op == "read":
            return {"bytes": int(code + rows * case["dim"] * es), "flops": rows * case["dim"]}
        return {"bytes": int(code + rows * case["dim"] * (es + 2)), "flops": 4 * rows * case["dim"]}
    t, hq, hk, d = case["draft"], case["heads"], case["kv_heads"], case["dim"]
    kv = sum(n + t for n in _lens(case))
    return {"bytes": int(2 * kv * hk * (d * CODE_BYTES[case["fmt"]] + 4) +
                         case["batch"] * t * hq * (4 * d + 4)),
            "flops": 4 * hq * t * d * kv}


# ------------------------------------------------------------------ inputs

def _levels():
    """bf16((q/15)^(1/alpha)), q = 0..15, as float32."""
    a = float(np.float32(ALPHA))
    g = [(q / 15.0) ** (1.0 / a) for q in range(16)]
    return torch.tensor(g, dtype=torch.float64).to(torch.bfloat16).float().to(DEV)


def _points():
    """The smallest float32 u whose code is k, k = 1..15."""
    a = float(np.float32(ALPHA))
    t = ((np.arange(1, 16) - 0.5) / 15.0) ** (1.0 / a)
    f = t.astype(np.float32)
    return torch.from_numpy(np.where(f < t, np.nextafter(f, np.float32(2)), f)).to(DEV)


def _code_shape(fmt, dim):
    return {"bf16": (torch.bfloat16, dim), "fp8": (torch.float8_e4m3fn, dim), "opq4": (torch.int32, dim // 8)}[fmt]


def _new_side(pages, heads, page, dim, fmt):
    dt, words = _code_shape(fmt, dim)
    codes = torch.zeros((pages, heads, page, words), dtype=torch.uint8 if fmt == "fp8" else dt, device=DEV)
    return {"codes": codes.view(dt) if fmt == "fp8" else codes,
            "sign": torch.zeros((pages, heads, page, dim // 32), dtype=torch.int32, device=DEV) if fmt == "opq4" else None,
            "scale": torch.zeros((pages, heads, page), dtype=torch.float32, device=DEV)}


def _normal(gen, shape, dim):
    """Values of a projection: normal, a few channels of the head much larger than the rest."""
    x = torch.randn(shape, generator=gen, device=DEV)
    gain = torch.ones(dim, device=DEV)
    gain[torch.randint(0, dim, (dim // 32,), generator=gen, device=DEV)] = 4.0
    return x.mul_(gain)


def _rows(gen, n, dim, fmt, points):
    """(codes, sign, scale) of n rows of a filled cache."""
    parts = []
    for at in range(0, n, 1 << 19):
        parts.append(_encode(_normal(gen, (min(1 << 19, n - at), dim), dim), fmt, points))
    cat = [None if p[0] is None else torch.cat([q.view(torch.uint8) if q.dtype == torch.float8_e4m3fn else q for q in p])
           for p in zip(*parts)]
    return (cat[0].view(torch.float8_e4m3fn) if fmt == "fp8" else cat[0]), cat[1], cat[2]


def _tree(rng, batch, draft):
    """Mask words of random trees: token i hangs under an earlier token or the prefix and
    sees itself and the tokens above it."""
    bits = np.zeros((batch, draft, draft), bool)
    for b in range(batch):
        for i in range(draft):
            parent = int(rng.integers(max(-1, i - 6), i))
            if parent >= 0:
                bits[b, i] = bits[b, parent]
            bits[b, i, i] = True
    words = np.zeros((batch, draft, -(-draft // 32)), np.uint32)
    for j in range(draft):
        words[:, :, j // 32] |= bits[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(words.view(np.int32)).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    if op == "rotary":
        t, axes, pairs = case["tokens"], case["axes"], case["rot"] // 2
        sections = [pairs] if axes == 1 else [pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8]
        freq = np.concatenate([10000.0 ** (-np.arange(n) / n) for n in sections])
        angle = np.arange(case["table"], dtype=np.float64)[:, None] * freq
        table = torch.from_numpy(np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)).to(DEV)
        if axes == 1 and t > 64:  # a sequence from somewhere on
            start = int(rng.integers(0, max(1, case["table"] - t)))
            pos = (start + np.arange(t))[:, None] % case["table"]
        elif axes == 1:
            pos = rng.integers(0, case["table"], (t, 1))
        else:  # a grid of image tokens after some text
            side = max(1, math.isqrt(t))
            pos = np.stack([np.full(t, int(rng.integers(0, 512))), np.arange(t) // side, np.arange(t) % side], 1)
        x = torch.randn((t, case["row_heads"], case["dim"]), generator=gen, device=DEV).to(TYPES[case["dtype"]])
        return {"case": case, "x": x[:, :case["heads"]], "table": table, "sections": sections,
                "positions": torch.from_numpy(pos.astype(np.int32)).to(DEV)}
    points, levels = _points(), _levels()
    fmt, dim, page = case["fmt"], case["dim"], case["page"]
    if op in ("write", "read"):
        t, heads = case["tokens"], case["heads"]
        pages = -(-t // page) + 1
        order = torch.from_numpy(rng.permutation(pages)).to(DEV)
        if t <= 64:  # one new token in each of t sequences
            pages = t + 1
            slots = torch.from_numpy(rng.permutation(pages)[:t] * page + rng.integers(0, page, t)).to(DEV)
        else:        # one sequence, page after page
            first = int(rng.integers(0, page))
            at = torch.arange(t, device=DEV) + min(first, pages * page - t)
            slots = order[at // page] * page + at % page
        s = {"case": case, "slots": slots.to(torch.int32), "points": points, "levels": levels}
        if op == "write":
            s["k"], s["v"] = (_normal(gen, (t, heads, dim), dim).to(TYPES[case["dtype"]]) for _ in range(2))
            s["sides"] = [_new_side(pages, heads, page, dim, fmt) for _ in range(2)]
            return s
    else:
        lens, draft, heads = _lens(case), case["draft"], case["kv_heads"]
        per = -(-(max(lens) + draft) // page)
        pages = case["batch"] * per + 1
        ids = rng.permutation(pages)[:case["batch"] * per].reshape(case["batch"], per)
        q = torch.randn((case["batch"], draft, (case["heads"] + 2 * heads) * dim), generator=gen, device=DEV)
        s = {"case": case, "points": points, "levels": levels, "longest": max(lens),
             "q": q.to(torch.bfloat16)[..., :case["heads"] * dim].unflatten(-1, (case["heads"], dim)),
             "page_table": torch.from_numpy(ids.astype(np.int32)).to(DEV),
             "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
             "mask": _tree(rng, case["batch"], draft) if draft > 1 else None}
    s["sides"] = []
    for _ in range(2):
        codes, sign, scale = _rows(gen, pages * heads * page, dim, fmt, points)
        s["sides"].append({"codes": codes.unflatten(0, (pages, heads, page)),
                           "sign": None if sign is None else sign.unflatten(0, (pages, heads, page)),
                           "scale": scale.unflatten(0, (pages, heads, page))})
    return s


# ------------------------------------------------------------------ the plain forms

def _encode(x, fmt, points):
    """(codes, sign, scale) of rows x [..., dim]."""
    x = x.float()
    if fmt == "bf16":
        return x.to(torch.bfloat16), None, torch.ones_like(x[..., 0])
    m = x.abs().amax(-1)
    if fmt == "fp8":
        s = m / torch.full_like(m, 448.0)  # a quotient by a tensor is rounded once; by a number it is a product
        y = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
        return y.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), None, s
    u = torch.where(m[..., None] > 0, x.abs() / m[..., None], torch.zeros_like(x))
    q = torch.bucketize(u, points, out_int32=True, right=True)
    shift = 4 * torch.arange(8, device=x.device, dtype=torch.int32)
    packed = (q.unflatten(-1, (-1, 8)) << shift).sum(-1).to(torch.int32)
    bit = torch.arange(32, device=x.device, dtype=torch.int32)
    sign = ((x < 0).to(torch.int32).unflatten(-1, (-1, 32)) << bit).sum(-1).to(torch.int32)
    return packed, sign, m


def _decode(codes, sign, scale, levels):
    """float32 values of stored rows."""
    if sign is None:
        return codes.float() * scale[..., None]
    shift = 4 * torch.arange(8, device=codes.device, dtype=torch.int32)
    q = ((codes[..., None] >> shift) & 15).flatten(-2)
    bit = torch.arange(32, device=codes.device, dtype=torch.int32)
    neg = ((sign[..., None] >> bit) & 1).flatten(-2)
    g = levels[q]
    return torch.where(neg != 0, -g, g) * scale[..., None]


def _turned(state):
    c, x, pairs = state["case"], state["x"].float(), state["table"].shape[1]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=x.device),
                                   torch.tensor(state["sections"], device=x.device), output_size=pairs)
    at = state["positions"].long()[:, axis]                                  # [tokens, pairs]
    cs = state["table"][at, torch.arange(pairs, device=x.device)].unsqueeze(1)
    cos, sin = cs[..., 0], -cs[..., 1] if c["grad"] else cs[..., 1]
    rot = 2 * pairs
    a, b = (x[..., :pairs], x[..., pairs:rot]) if c["layout"] == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    p, q = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat((p, q), -1) if c["layout"] == "half" else torch.stack((p, q), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).to(state["x"].dtype)


def _at_slots(side, slots, levels):
    page = side["scale"].shape[2]
    p, o = slots.long() // page, slots.long() % page
    codes = side["codes"].view(torch.uint8)[p, :, o].view(torch.float8_e4m3fn) \
        if side["codes"].dtype == torch.float8_e4m3fn else side["codes"][p, :, o]
    return _decode(codes, None if side["sign"] is None else side["sign"][p, :, o], side["scale"][p, :, o], levels)


def _written(side, x, slots, fmt, points):
    page = side["scale"].shape[2]
    p, o = slots.long() // page, slots.long() % page
    codes, sign, scale = _encode(x, fmt, points)
    if fmt == "fp8":
        side["codes"].view(torch.uint8)[p, :, o] = codes.view(torch.uint8)
    else:
        side["codes"][p, :, o] = codes
    if sign is not None:
        side["sign"][p, :, o] = sign
    side["scale"][p, :, o] = scale


def _gathered(side, table, levels):
    """float32 [batch, heads, tokens, dim] of every sequence's pages."""
    ids = table.long()
    codes = side["codes"].view(torch.uint8)[ids].view(torch.float8_e4m3fn) \
        if side["codes"].dtype == torch.float8_e4m3fn else side["codes"][ids]
    v = _decode(codes, None if side["sign"] is None else side["sign"][ids], side["scale"][ids], levels)
    return v.transpose(1, 2).flatten(2, 3)


def _attended(state):
    c, q = state["case"], state["q"].float()
    b, t, hq, d = q.shape
    hk = c["kv_heads"]
    k = _gathered(state["sides"][0], state["page_table"], state["levels"])
    v = _gathered(state["sides"][1], state["page_table"], state["levels"])
    j = torch.arange(k.shape[2], device=q.device)
    lens = state["lens"].long()
    drafted = (j - lens[:, None]).clamp(0, t - 1)                              # [b, kv]
    if state["mask"] is None:
        seen = torch.ones((b, t, j.numel()), dtype=torch.bool, device=q.device)
    else:
        bits = ((state["mask"][..., None] >> torch.arange(32, device=q.device, dtype=torch.int32)) & 1).flatten(-2) != 0
        seen = torch.gather(bits, 2, drafted[:, None].expand(b, t, j.numel()))
    seen = (seen | (j < lens[:, None])[:, None]) & (j < lens[:, None] + t)[:, None]
    rows = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    s = torch.matmul(rows, k.transpose(2, 3).contiguous()).mul_(d ** -0.5).unflatten(2, (t, hq // hk))
    s.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (t, hq // hk))
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, float("-inf")))[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).flatten(2, 3).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).flatten(2, 3).contiguous()}


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _run_own(state, c, op)
    if op == "rotary":
        return _turned(state)
    if op == "attention":
        return _attended(state)
    k, v = state["sides"]
    if op == "read":
        out = TYPES[c["dtype"]]
        return {"k": _at_slots(k, state["slots"], state["levels"]).to(out),
                "v": _at_slots(v, state["slots"], state["levels"]).to(out)}
    _written(k, state["k"], state["slots"], c["fmt"], state["points"])
    _written(v, state["v"], state["slots"], c["fmt"], state["points"])
    return {"k": _at_slots(k, state["slots"], state["levels"]).to(torch.bfloat16),
            "v": _at_slots(v, state["slots"], state["levels"]).to(torch.bfloat16),
            "k_scale": k["scale"], "v_scale": v["scale"]}


def _run_own(state, c, op):
    from w4a16_linear_amd import attention as A

    if op == "rotary":
        call = A.rotary_backward if c["grad"] else A.rotary
        return call(state["x"], state["positions"], state["table"], layout=c["layout"], sections=state["sections"])
    k, v = state["sides"]
    cache = A.PagedCache(c["fmt"], ALPHA, k["codes"], k["sign"], k["scale"], v["codes"], v["sign"], v["scale"])
    if op == "attention":
        out, lse = A.tree_attention(state["q"], cache, state["page_table"], state["lens"], mask=state["mask"],
                                    max_len=state["longest"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "read":
        got = A.cache_read(cache, state["slots"], out_dtype=TYPES[c["dtype"]])
        return {"k": got[0], "v": got[1]}
    A.cache_write(cache, state["k"], state["v"], state["slots"])
    got = A.cache_read(cache, state["slots"])
    return {"k": got[0], "v": got[1], "k_scale": k["scale"], "v_scale": v["scale"]}


# ------------------------------------------------------------------ in 64 bits

def _round_to(x, bits, lowest):
    """x (float64) to `bits` significant bits, halves to even, steps no finer than at 2^lowest."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** (lowest - 60)))).clamp_min(lowest)
    step = torch.exp2(e - (bits - 1))
    return torch.round(x / step) * step


def _exact_levels():
    a = float(np.float32(ALPHA))
    q = torch.arange(16, dtype=torch.float64, device=DEV) / 15.0
    return _round_to(q ** (1.0 / a), 8, -100)


def _exact_rows(x, fmt):
    """(values, scale) that rows x [..., dim] read back as, in float64."""
    x = x.double()
    if fmt == "bf16":
        return _round_to(x, 8, -120), torch.ones_like(x[..., 0])
    m = x.abs().amax(-1)
    if fmt == "fp8":
        s = (m / 448.0).float().double()
        r = (x / s[..., None].clamp_min(1e-300)).float().double()
        return _round_to(r, 4, -6) * s[..., None], s
    u = (x.abs() / m[..., None].clamp_min(1e-300)).float().double()
    q = torch.floor(15.0 * u ** float(np.float32(ALPHA)) + 0.5).long()
    return torch.sign(x) * _exact_levels()[q] * m[..., None], m


def _exact_stored(side, index):
    """float64 [heads, n, dim] of the rows of the pages `index`, in order."""
    codes, scale = side["codes"], side["scale"][index].double()
    if side["sign"] is None:
        if codes.dtype == torch.float8_e4m3fn:
            byte = codes.view(torch.uint8)[index].double()
            mag, neg = byte % 128, byte >= 128
            e, f = torch.floor(mag / 8), mag % 8
            g = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - 7), f * 2.0 ** -9)
            g = torch.where(neg, -g, g)
        else:
            g = codes[index].double()
    else:
        q = torch.stack([(codes[index] // 16 ** i) % 16 if i < 7 else (codes[index] >> 28) % 16 for i in range(8)], -1).flatten(-2)
        n = torch.stack([(side["sign"][index] >> i) % 2 for i in range(32)], -1).flatten(-2)
        g = _exact_levels()[q.long()] * (1 - 2 * n.double())
    return (g * scale[..., None]).transpose(0, 1).flatten(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        x, pairs = s["x"].double(), case["rot"] // 2
        axis = np.repeat(np.arange(case["axes"]), s["sections"])
        c = torch.stack([s["table"][s["positions"][:, axis[i]].long(), i].double() for i in range(pairs)], 1)
        z = torch.complex(c[..., 0], -c[..., 1] if case["grad"] else c[..., 1])[:, None]
        out = x.clone()
        lo, hi = (slice(0, pairs), slice(pairs, 2 * pairs)) if case["layout"] == "half" else \
            (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))
        w = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * z
        out[..., lo], out[..., hi] = w.real, w.imag
        return out
    if op == "write":
        k, ks = _exact_rows(s["k"], case["fmt"])
        v, vs = _exact_rows(s["v"], case["fmt"])
        page, scales = case["page"], []
        for side, new in zip(s["sides"], (ks, vs)):
            scale = side["scale"].double()
            scale[s["slots"].long() // page, :, s["slots"].long() % page] = new
            scales.append(scale)
        return {"k": k, "v": v, "k_scale": scales[0], "v_scale": scales[1]}
    if op == "read":
        got = []
        for side in s["sides"]:
            rows = _exact_stored(side, torch.arange(side["scale"].shape[0], device=DEV))
            got.append(rows[:, s["slots"].long()].transpose(0, 1).contiguous())
        return {"k": got[0], "v": got[1]}
    t, hq, hk, d = case["draft"], case["heads"], case["kv_heads"], case["dim"]
    outs, lses = [], []
    for b, n in enumerate(_lens(case)):
        pages = s["page_table"][b, :-(-(n + t) // case["page"])].long()
        k, v = (_exact_stored(side, pages)[:, :n + t] for side in s["sides"])
        q = s["q"][b].double().permute(1, 0, 2)                               # [hq, t, d]
        hide = torch.zeros((t, n + t), dtype=torch.bool, device=DEV)
        if t > 1:
            words = s["mask"][b].cpu().numpy().view(np.uint32)
            hide[:, n:] = torch.from_numpy(np.array(
                [[not (int(words[i, j // 32]) >> (j % 32)) & 1 for j in range(t)] for i in range(t)])).to(DEV)
        o = torch.empty((hq, t, d), dtype=torch.float64, device=DEV)
        lse = torch.empty((hq, t), dtype=torch.float64, device=DEV)
        for h in range(hk):
            of = slice(h * (hq // hk), (h + 1) * (hq // hk))
            w = (q[of].reshape(-1, d) @ k[h].T).reshape(hq // hk, t, n + t) / math.sqrt(d)
            w = w.masked_fill(hide, -math.inf)
            lse[of] = torch.logsumexp(w, -1)
            o[of] = (torch.exp(w - lse[of][..., None]).reshape(-1, n + t) @ v[h]).reshape(hq // hk, t, d)
        outs.append(o.transpose(0, 1))
        lses.append(lse.T)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
