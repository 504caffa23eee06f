"""The operators of many requests (low-rank adapters and the gradient through a quantized
projection, verification of drafted tokens, pages of a cache forked and moved): the workloads
they are measured on, and their plain forms.

`run` computes an operator in elementary torch operations in float32 (float64 at borders) where
`own` is false, and calls the framework (w4a16_linear_amd.adapters and .attention) where it is
true.  `exact` gives the same outputs in float64 or exact integers from the definitions, written
apart from the plain forms.

Definitions (the framework's modules document them for users):
  adapters  down [adapters, rank, in], up [adapters, rank, out], scale [adapters], index [tokens]:
            out_t = y_t + s_i U_i^T (D_i x_t) with i = index[t]; a token whose index names no
            adapter keeps its y.  Backward, from dy: e_t = s_i U_i dy_t, h_t = D_i x_t;
            dx_t = (dx of the projection)_t + D_i^T e_t, dD_i = sum_t e_t x_t^T,
            dU_i = sum_t s_i h_t dy_t^T.
  linear    dx = dy W', W' = +-bfloat16(G_q m) of 4-bit codes (opq_dequantize's values).
  verify    token 0 of a sequence's draft is certain; row t of the target's probabilities p is the
            distribution after token t.  From node 0 on, the children of the node are tested in
            index order: with draft probabilities q (a chain) a token x is kept if u q(x) < p(x),
            without (a tree) if u Z < p(x), Z = 1 less the p of the siblings tested before.  At the
            last kept node `next` is drawn with u_0: from p; from max(p - q, 0) if a token drawn from
            q was refused; from p without the refused tokens in a tree.  It is the lowest token
            whose cumulative weight exceeds u_0 times the weights' sum.
  pages     a page table names pages of a cache; a page that no entry names is free.
            fork: row i of the new table holds what row parents[i] names of its lens tokens; a last,
            partly filled page stays with the first row that names it, unless a row names it as a
            full one; each other row gets the lowest free page, and a pair (src, dst) to copy.
            resize: rows keep the entries that their tokens need and take the lowest free pages for
            those they lack, row by row.  compact: used pages move to the lowest ids, the k-th used
            page past them to the k-th free place.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ALPHA = 0.73
HIDDEN, QKV, FFN, FFN_UPGATE = 3840, 11520, 10240, 20480
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"bf16": (torch.bfloat16, 2.0), "fp8": (torch.uint8, 1.0), "opq4": (torch.int32, 0.625)}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user with an adapter of their own on the output projection, one new token
        dict(name="adapters: one token", op="adapters", tokens=1, k=HIDDEN, n=HIDDEN, rank=8,
             adapters=4, requests=1, dtype="bf16", out="bf16"),
        # 48 users, one new token each, adapters out of 64, on the fused QKV projection
        dict(name="adapters: one token each", op="adapters", tokens=48, k=HIDDEN, n=QKV, rank=16,
             adapters=64, requests=48, dtype="bf16", out="bf16"),
        # the prompts of several requests, ranks padded to the largest, on the FFN's up and gate projection
        dict(name="adapters: prompts", op="adapters", tokens=4096, k=HIDDEN, n=FFN_UPGATE, rank=64,
             adapters=16, requests=7, dtype="bf16", out="bf16"),
        # a training step of one adapter on the fused QKV projection
        dict(name="adapters' gradients: one", op="gradients", tokens=4096, k=HIDDEN, n=QKV, rank=16,
             adapters=1, requests=1, dtype="bf16", out="bf16"),
        # several adapters trained at once on the FFN's down projection, sums kept in 32 bits, odd length
        dict(name="adapters' gradients: several", op="gradients", tokens=2047, k=FFN, n=HIDDEN, rank=32,
             adapters=5, requests=9, dtype="bf16", out="f32"),
        # the gradient through the quantized output projection, a short odd batch, one max a group of 128
        dict(name="projection's gradient: short", op="linear", tokens=333, k=HIDDEN, n=HIDDEN, group=128,
             out="bf16"),
        # the gradient through the quantized QKV projection
        dict(name="projection's gradient", op="linear", tokens=4096, k=HIDDEN, n=QKV, group=0, out="bf16"),
        # one user, a tree of candidates
        dict(name="verify: one tree", op="verify", batch=1, draft=24, vocab=32000, tree=True, dtype="f32"),
        # a serving batch, chains from a draft model
        dict(name="verify: chains", op="verify", batch=48, draft=6, vocab=131072, tree=False, dtype="f32"),
        # four users' beams of eight, forked after a step, with the copies of their last pages
        dict(name="pages: beams forked", op="fork", rows=32, columns=24, beams=8, page=64, pages=512,
             heads=8, dim=128, fmt="fp8"),
        # a large pool: many samples of some prompts; new tables, few copies
        dict(name="pages: many rows forked", op="fork", rows=1024, columns=300, beams=16, page=16,
             pages=65536, heads=1, dim=64, fmt="fp8"),
        # a cache drawn together before memory is handed back
        dict(name="pages: compacted", op="compact", rows=128, columns=40, page=64, pages=4096, used=2100,
             moved=900, heads=8, dim=128, fmt="opq4"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for case in listed():
        w, m = work(case), most.setdefault(case["op"], {"bytes": 0, "flops": 0})
        for key in m:
            m[key] = max(m[key], w[key])
    while True:
        op = rng.choice(("adapters", "adapters", "gradients", "gradients", "linear", "verify", "verify", "fork", "compact"))
        if op in ("adapters", "gradients"):
            tokens = _log(rng, 1, 8192)
            case = dict(op=op, tokens=tokens, k=32 * _log(rng, 8, 320), n=8 * _log(rng, 32, 2560),
                        rank=rng.choice((8, 16, 16, 24, 32, 64, 128)), adapters=_log(rng, 1, 64),
                        requests=min(tokens, _log(rng, 1, 64)), dtype=rng.choice(("bf16", "bf16", "f32")),
                        out=rng.choice(("bf16", "f32")))
        elif op == "linear":
            k = 256 * _log(rng, 1, 40)
            case = dict(op=op, tokens=_log(rng, 1, 4096), k=k, n=8 * _log(rng, 16, 2560),
                        group=rng.choice((0, 0, 0, 32, 128, 256)), out=rng.choice(("bf16", "f32")))
        elif op == "verify":
            case = dict(op=op, batch=_log(rng, 1, 64), draft=rng.choice((1, 2, 3, 5, 6, 9, 16, 33, 64)),
                        vocab=_log(rng, 500, 160000), tree=rng.random() < 0.5, dtype=rng.choice(("f32", "f32", "bf16")))
            if case["batch"] * case["draft"] * case["vocab"] > 48 * 6 * 131072:
                continue
        else:
            beams = rng.choice((1, 2, 4, 5, 8, 16))
            case = dict(op=op, rows=beams * _log(rng, 1, 64), columns=_log(rng, 3, 256), page=rng.choice((16, 32, 64, 128)),
                        heads=rng.choice((1, 2, 4, 5, 8)), dim=rng.choice((64, 128, 256)),
                        fmt=rng.choice(("bf16", "fp8", "opq4")))
            if op == "fork":
                need = case["rows"] // beams * case["columns"] + 9 * case["rows"]
                case.update(beams=beams, pages=need + _log(rng, 1, 4096))
            else:
                used = _log(rng, 2, max(3, case["rows"] * case["columns"]))
                case.update(pages=used + _log(rng, 1, 4096), used=used)
                case["moved"] = min(used, case["pages"] - used, _log(rng, 1, used))
            if case["pages"] * case["heads"] * case["page"] * (case["dim"] * CODES[case["fmt"]][1] + 4) > 200e6:
                continue
        w = work(case)
        if all(w[key] <= most[op][key] for key in w):
            return case


def _copies(case):
    """Pages a fork copies: in each group of beams half of the rows (rounded down) have a parent
    that another row has too."""
    return (case["rows"] // case["beams"]) * (case["beams"] // 2)


def work(case):
    op = case["op"]
    if op in ("adapters", "gradients"):
        m, k, n, r = case["tokens"], case["k"], case["n"], case["rank"]
        used = min(case["adapters"], case["requests"])
        size, out = (2 if case[key] == "bf16" else 4 for key in ("dtype", "out"))
        if op == "adapters":
            return {"bytes": 2 * m * k + m * n * (size + out) + 2 * used * r * (k + n) + 4 * m,
                    "flops": 2 * m * r * (k + n)}
        return {"bytes": 2 * m * (k + n) + 2 * m * k * size + 2 * used * r * (k + n) +
                         case["adapters"] * r * (k + n) * out + 4 * m,
                "flops": 2 * m * r * (3 * k + 2 * n)}
    if op == "linear":
        m, k, n = case["tokens"], case["k"], case["n"]
        scales = 4 * n if case["group"] == 0 else 2 * n * (k // case["group"])
        return {"bytes": int(0.625 * n * k) + scales + 2 * m * n + m * k * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    if op == "verify":
        rows = case["batch"] * (1 if case["tree"] or case["draft"] == 1 else 2)
        return {"bytes": rows * case["vocab"] * (4 if case["dtype"] == "f32" else 2) + 16 * case["batch"] * case["draft"],
                "flops": rows * case["vocab"]}
    moved = _copies(case) if op == "fork" else case["moved"]
    row = case["dim"] * CODES[case["fmt"]][1] + 4
    return {"bytes": int(2 * moved * 2 * case["heads"] * case["page"] * row + 8 * case["rows"] * case["columns"]),
            "flops": case["rows"] * case["columns"]}


# ------------------------------------------------------------------ inputs

def _points():
    """The smallest float32 u whose code is q, q = 1..15."""
    t = ((np.arange(1, 16) - 0.5) / 15.0) ** (1.0 / float(np.float32(ALPHA)))
    f = t.astype(np.float32)
    return torch.from_numpy(np.where(f < t, np.nextafter(f, np.float32(2)), f)).to(DEV)


def _runs(rng, tokens, requests):
    """Lengths of `requests` requests that make up `tokens` tokens, every one at least 1."""
    cuts = np.sort(rng.choice(np.arange(1, tokens), requests - 1, replace=False)) if requests > 1 else np.zeros(0, int)
    return np.diff(np.concatenate(([0], cuts, [tokens])))


def _pool(rng, case):
    """A page table and lengths of groups of beams: each group shares a prompt's pages, its
    beams have pages of their own after them.  All beams of a group are equally long."""
    rows, columns, beams, page = case["rows"], case["columns"], case["beams"], case["page"]
    table = np.full((rows, columns), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    ids = rng.permutation(case["pages"])
    at = 0
    for g in range(rows // beams):
        held = int(rng.integers(max(1, columns // 2), columns))      # one column is left for the next token
        shared = held - int(rng.integers(1, min(held, 8) + 1))       # the last page is a beam's own
        length = (held - 1) * page + int(rng.integers(1, page))      # and partly filled
        prompt = ids[at:at + shared]
        at += shared
        for b in range(beams):
            table[g * beams + b, :shared] = prompt
            table[g * beams + b, shared:held] = ids[at:at + held - shared]
            at += held - shared
            lens[g * beams + b] = length
    return table, lens


def _cache(gen, case):
    """Keys' and values' codes, signs and scales of a filled cache."""
    kind, words = CODES[case["fmt"]][0], {"bf16": case["dim"], "fp8": case["dim"], "opq4": case["dim"] // 8}[case["fmt"]]
    lead = (case["pages"], case["heads"], case["page"])
    sides = []
    for _ in range(2):
        if kind == torch.bfloat16:
            codes = torch.randn(lead + (words,), generator=gen, device=DEV).to(kind)
        elif kind == torch.uint8:
            codes = torch.randint(0, 126, lead + (words,), generator=gen, device=DEV, dtype=kind)
        else:
            codes = torch.randint(-2 ** 31, 2 ** 31, lead + (words,), generator=gen, device=DEV, dtype=kind)
        sign = torch.randint(-2 ** 31, 2 ** 31, lead + (case["dim"] // 32,), generator=gen, device=DEV,
                             dtype=torch.int32) if case["fmt"] == "opq4" else None
        sides.append({"codes": codes, "sign": sign, "scale": torch.rand(lead, generator=gen, device=DEV) + 0.5})
    return sides


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if op in ("adapters", "gradients"):
        m, k, n, r, count = case["tokens"], case["k"], case["n"], case["rank"], case["adapters"]
        runs = _runs(rng, m, case["requests"])
        ids = np.concatenate([rng.permutation(count) for _ in range(-(-len(runs) // count))])[:len(runs)].astype(np.int32)
        if op == "adapters" and len(runs) > 4:
            ids[rng.integers(0, len(runs), len(runs) // 8)] = -1      # some requests use the base alone
        gain = torch.ones(k, device=DEV)
        gain[torch.randint(0, k, (k // 128,), generator=gen, device=DEV)] = 8.0
        s = {"case": case, "x": (normal(m, k) * gain).to(torch.bfloat16),
             "down": (normal(count, r, k) * k ** -0.5).to(torch.bfloat16),
             "up": (normal(count, r, n) * 0.05).to(torch.bfloat16),
             "scale": torch.rand(count, generator=gen, device=DEV) * 1.5 + 0.5,
             "index": torch.from_numpy(np.repeat(ids, runs)).to(DEV),
             "runs": [(int(i), int(e - l), int(e)) for i, l, e in zip(ids, runs, np.cumsum(runs))]}
        if op == "adapters":
            s["y"] = normal(m, n).to(TYPES[case["dtype"]])
        else:
            s["dy"] = (normal(m, n) * 0.01).to(torch.bfloat16)
            s["dx"] = (normal(m, k) * 0.01).to(TYPES[case["dtype"]])
        return s
    if op == "linear":
        m, k, n, group = case["tokens"], case["k"], case["n"], case["group"]
        w = normal(n, k) * 0.02
        w = w.to(torch.bfloat16).float()
        top = w.abs().view(n, -1, group or k).amax(-1)
        if group:
            top = top.half()
        u = w.abs().view(n, -1, group or k) / top.float()[..., None]
        q = torch.bucketize(u, _points(), out_int32=True, right=True).view(n, k)
        nibble = torch.arange(8, device=DEV, dtype=torch.int32) * 4
        bit = torch.arange(32, device=DEV, dtype=torch.int32)
        return {"case": case, "dy": (normal(m, n) * 0.01).to(torch.bfloat16),
                "packed": (q.view(n, -1, 8) << nibble).sum(-1).to(torch.int32),
                "sign": ((w < 0).to(torch.int32).view(n, -1, 32) << bit).sum(-1).to(torch.int32),
                "scale": top if group else top[:, 0].contiguous()}
    if op == "verify":
        b, t, v = case["batch"], case["draft"], case["vocab"]
        logits = normal(b, t, v) * 3.0
        p = torch.softmax(logits, -1)
        parents = np.tile(np.arange(-1, t - 1, dtype=np.int32), (b, 1))
        s = {"case": case, "uniforms": torch.rand((b, t), generator=gen, device=DEV)}
        if case["tree"]:
            for i in range(1, t):
                parents[:, i] = rng.integers(max(0, i - 8), i, b)
            s["parents"] = torch.from_numpy(parents).to(DEV)
            # candidates: likely tokens of the node they hang under
            likely = torch.topk(p, min(v, 16), -1).indices
            rank = torch.from_numpy(rng.integers(0, min(v, 16), (b, t))).to(DEV)
            node = s["parents"].long().clamp_min(0)
            tokens = likely[torch.arange(b, device=DEV)[:, None], node, rank]
        else:
            q = torch.softmax(logits[:, :max(0, t - 1)].add_(normal(b, max(0, t - 1), v)), -1).to(TYPES[case["dtype"]])
            race = torch.empty_like(q, dtype=torch.float32).exponential_(generator=gen)
            tokens = torch.cat((torch.randint(0, v, (b, 1), generator=gen, device=DEV), (q.float() / race).argmax(-1)), 1)
            s["q"] = q
        s["p"] = p.to(TYPES[case["dtype"]])
        s["tokens"] = tokens.to(torch.int32)
        return s
    s = {"case": case, "sides": _cache(gen, case)}
    if op == "fork":
        table, lens = _pool(rng, case)
        parents = np.zeros(case["rows"], np.int32)
        for g in range(case["rows"] // case["beams"]):
            # the worse half of the beams goes, each of the better half's best goes on twice
            order = rng.permutation(case["beams"])
            keep = case["beams"] - case["beams"] // 2
            parents[g * case["beams"]:][:case["beams"]] = g * case["beams"] + rng.permutation(
                np.concatenate((order[:keep], order[:case["beams"] - keep])))
        s.update(table=torch.from_numpy(table).to(DEV), lens=torch.from_numpy(lens).to(DEV),
                 parents=torch.from_numpy(parents).to(DEV))
        return s
    used, moved, pages = case["used"], case["moved"], case["pages"]
    ids = np.concatenate((rng.permutation(used)[:used - moved], used + rng.permutation(pages - used)[:moved]))
    table = np.full(case["rows"] * case["columns"], -1, np.int32)
    places = rng.permutation(table.size)
    table[places[:used]] = rng.permutation(ids)                        # every used page once
    extra = places[used:used + used // 4]
    table[extra] = rng.choice(ids, extra.size)                         # and some of them again: shared
    s["table"] = torch.from_numpy(table.reshape(case["rows"], case["columns"])).to(DEV)
    return s


# ------------------------------------------------------------------ the plain forms

def _adapted(s):
    c = s["case"]
    y, out = s["y"], TYPES[c["out"]]
    if c["tokens"] <= 64:                                              # a token each: gathered adapters
        at = s["index"].long().clamp_min(0)
        h = torch.matmul(s["down"][at].float(), s["x"].float()[:, :, None])
        d = torch.matmul(h.transpose(1, 2).contiguous(), s["up"][at].float())[:, 0]
        d = d * torch.where(s["index"] >= 0, s["scale"][at], torch.zeros_like(s["scale"][at]))[:, None]
        return (y.float() + d).to(out)
    parts = []
    for i, a, e in s["runs"]:                                          # request by request
        part = y[a:e].float()
        if i >= 0:
            h = torch.matmul(s["x"][a:e].float(), s["down"][i].float().T)
            part = part + torch.matmul(h * s["scale"][i], s["up"][i].float())
        parts.append(part.to(out))
    return torch.cat(parts)


def _gradients(s):
    c = s["case"]
    down, up = torch.zeros_like(s["down"], dtype=torch.float32), torch.zeros_like(s["up"], dtype=torch.float32)
    parts = []
    for i, a, e in s["runs"]:
        x, dy, w, v = s["x"][a:e].float(), s["dy"][a:e].float(), s["down"][i].float(), s["up"][i].float()
        h = torch.matmul(x, w.T) * s["scale"][i]
        g = torch.matmul(dy, v.T) * s["scale"][i]
        parts.append((s["dx"][a:e].float() + torch.matmul(g, w)).to(s["dx"].dtype))
        down[i] += torch.matmul(g.T, x)
        up[i] += torch.matmul(h.T, dy)
    return {"dx": torch.cat(parts), "down": down.to(TYPES[c["out"]]), "up": up.to(TYPES[c["out"]])}


def _through(s):
    c = s["case"]
    a = float(np.float32(ALPHA))
    levels = (torch.arange(16, device=DEV, dtype=torch.float64) / 15.0) ** (1.0 / a)
    nibble = torch.arange(8, device=DEV, dtype=torch.int32) * 4
    bit = torch.arange(32, device=DEV, dtype=torch.int32)
    q = ((s["packed"][..., None] >> nibble) & 15).flatten(1)
    neg = ((s["sign"][..., None] >> bit) & 1).flatten(1)
    top = s["scale"].double()[..., None]
    if c["group"]:
        top = top.expand(-1, -1, c["group"]).flatten(1)
    w = (levels[q] * top).to(torch.bfloat16).float()
    return torch.matmul(s["dy"].float(), torch.where(neg != 0, -w, w)).to(TYPES[c["out"]])


def _verified(s):
    c = s["case"]
    b, t, v = c["batch"], c["draft"], c["vocab"]
    p, tokens, u = s["p"], s["tokens"].long(), s["uniforms"].double()
    row = torch.arange(b, device=DEV)
    if not c["tree"]:
        at = tokens[:, 1:, None]
        keep = u[:, 1:] * torch.gather(s["q"], 2, at)[..., 0].double() < torch.gather(p[:, :t - 1], 2, at)[..., 0].double()
        more = keep.long().cumprod(1).sum(1)                           # drafted tokens kept
        step = torch.arange(t, device=DEV)
        kept = torch.where(step <= more[:, None], step, -1)
        w = p[row, more].double()
        if t > 1:
            q = s["q"][row, more.clamp_max(t - 2)].double()
            w = torch.where((more < t - 1)[:, None], (w - q).clamp_min(0), w)
        count = more + 1
    else:
        node = torch.zeros(b, dtype=torch.long, device=DEV)
        left = torch.ones(b, dtype=torch.float64, device=DEV)
        gone = torch.zeros((b, v), dtype=torch.bool, device=DEV)       # tokens refused at the node
        kept = torch.full((b, t), -1, dtype=torch.long, device=DEV)
        kept[:, 0] = 0
        count = torch.ones(b, dtype=torch.long, device=DEV)
        for i in range(1, t):
            x = tokens[:, i]
            here = s["parents"][:, i] == node
            px = torch.where(gone[row, x], 0.0, p[row, node, x].double())
            take = here & (u[:, i] * left < px)
            drop = here & ~take
            left = torch.where(take, 1.0, torch.where(drop, left - px, left))
            gone[row, x] |= drop
            gone &= ~take[:, None]
            node = torch.where(take, i, node)
            kept[row, torch.where(take, count, t - 1)] = torch.where(take, i, kept[row, torch.where(take, count, t - 1)])
            count = count + take
        w = p[row, node].double().masked_fill_(gone, 0.0)
    sums = w.cumsum(1)
    drawn = torch.searchsorted(sums, u[:, :1] * sums[:, -1:], right=True)[:, 0]
    last = (w > 0).long().cumsum(1).argmax(1)                          # where rounding left none
    return {"kept": kept.to(torch.int32), "count": count.to(torch.int32),
            "next": torch.minimum(drawn, last).to(torch.int32)}


def _lowest_free(named, pages):
    """Page ids, the free ones first in ascending order (`named`: ids in use, or `pages` for none)."""
    used = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
    used[named.flatten()] = 1
    return torch.argsort(used[:pages], stable=True)


def _copy(s, src, dst, named):
    """Copy pages src to dst (-1: none); in place of a pair without pages the last page that
    `named` names, so no destination, is copied onto itself."""
    still = named.max()
    src, dst = torch.where(src >= 0, src, still), torch.where(src >= 0, dst, still)
    for side in s["sides"]:
        for t in side.values():
            if t is not None:
                t[dst] = t[src]
    return [t for side in s["sides"] for t in side.values() if t is not None]


def _forked(s):
    c = s["case"]
    page, pages, rows = c["page"], c["pages"], c["rows"]
    lens = s["lens"][s["parents"].long()].long()
    column = torch.arange(c["columns"], device=DEV)
    table = torch.where(column * page < lens[:, None], s["table"][s["parents"].long()], -1).long()
    full = torch.where((column + 1) * page <= lens[:, None], table, -1)
    part = torch.div(lens, page, rounding_mode="floor")
    partial = lens % page != 0
    i = torch.arange(rows, device=DEV)
    mine = torch.where(partial, table[i, part.clamp_max(c["columns"] - 1)], pages)
    first = torch.full((pages + 1,), rows, dtype=torch.long, device=DEV).scatter_reduce_(0, mine, i, "amin")
    held = torch.zeros(pages + 1, dtype=torch.bool, device=DEV)
    held[torch.where(full >= 0, full, pages).flatten()] = True
    copy = partial & ((first[mine] != i) | held[mine]) & (mine < pages)
    kept = torch.where(table >= 0, table, pages)
    kept[i, part.clamp_max(c["columns"] - 1)] = torch.where(copy, pages, kept[i, part.clamp_max(c["columns"] - 1)])
    free = _lowest_free(kept, pages)
    fresh = free[(copy.long().cumsum(0) - 1).clamp_min(0)]
    at = part.clamp_max(c["columns"] - 1)
    table[i, at] = torch.where(copy, fresh, table[i, at])
    src, dst = torch.where(copy, mine, -1), torch.where(copy, fresh, -1)
    state = _copy(s, src, dst, torch.where(kept < pages, kept, 0))
    # one more token each
    need = torch.div(lens + page, page, rounding_mode="floor")          # ceil((lens + 1) / page)
    table = torch.where(column < need[:, None], table, -1)
    lack = (column < need[:, None]) & (table < 0)
    free = _lowest_free(torch.where(table >= 0, table, pages), pages)
    order = lack.flatten().long().cumsum(0) - 1
    table = torch.where(lack, free[order.clamp_min(0)].view_as(table), table)
    return [table.to(torch.int32), src.to(torch.int32), dst.to(torch.int32)] + state


def _compacted(s):
    c = s["case"]
    pages, table = c["pages"], s["table"].long()
    used = torch.zeros(pages + 1, dtype=torch.long, device=DEV)
    used[torch.where(table >= 0, table, pages).flatten()] = 1
    used = used[:pages]
    count = used.sum()
    ids = torch.arange(pages, device=DEV)
    beyond, hole = (used > 0) & (ids >= count), (used == 0) & (ids < count)
    room = min(pages // 2, table.numel())
    src = torch.full((pages + 1,), -1, dtype=torch.long, device=DEV)
    dst = src.clone()
    src[torch.where(beyond, beyond.long().cumsum(0) - 1, pages)] = ids
    dst[torch.where(hole, hole.long().cumsum(0) - 1, pages)] = ids
    src, dst = src[:room], dst[:room]
    to = torch.cat((ids, ids.new_full((1,), -1)))
    to[torch.where(src >= 0, src, pages)] = torch.where(src >= 0, dst, -1)
    table = to[torch.where(table >= 0, table, pages)]
    state = _copy(s, src, dst, s["table"].long())
    return [table.to(torch.int32), src.to(torch.int32), dst.to(torch.int32), count.view(1).to(torch.int32)] + state


PLAIN = {"adapters": _adapted, "gradients": _gradients, "linear": _through, "verify": _verified, "fork": _forked,
         "compact": _compacted}


def run(state):
    if own:
        return _run_own(state, state["case"])
    return PLAIN[state["case"]["op"]](state)


def _run_own(s, c):
    op = c["op"]
    if op in ("adapters", "gradients", "linear"):
        from w4a16_linear_amd import adapters as L
        from w4a16_linear_amd import opq

        if op == "linear":
            w = opq.GroupedWeight(s["packed"], s["sign"], s["scale"], c["group"]) if c["group"] else \
                opq.QuantizedWeight(s["packed"], s["sign"], s["scale"])
            return L.linear_backward(s["dy"], w, ALPHA, out_dtype=TYPES[c["out"]])
        stack = L.Adapters(s["down"], s["up"], s["scale"])
        if op == "adapters":
            return L.lowrank_add(s["y"], s["x"], stack, s["index"], out_dtype=TYPES[c["out"]])
        dx, down, up = L.lowrank_backward(s["dy"], s["x"], stack, s["index"], dx=s["dx"], grad_dtype=TYPES[c["out"]])
        return {"dx": dx, "down": down, "up": up}
    from w4a16_linear_amd import attention as A

    if op == "verify":
        kept, count, drawn = A.verify_drafts(s["p"], s["tokens"], s["uniforms"], draft_probs=s.get("q"),
                                             parents=s.get("parents"))
        return {"kept": kept, "count": count, "next": drawn}
    k, v = s["sides"]
    codes = [side["codes"].view(torch.float8_e4m3fn) if c["fmt"] == "fp8" else side["codes"] for side in (k, v)]
    cache = A.PagedCache(c["fmt"], ALPHA, codes[0], k["sign"], k["scale"], codes[1], v["sign"], v["scale"])
    state = [t for side in s["sides"] for t in side.values() if t is not None]
    if op == "fork":
        table, lens, src, dst, _ = A.pages_fork(s["table"], s["lens"], s["parents"], c["pages"], c["page"])
        A.cache_copy_pages(cache, src, dst)
        table, _ = A.pages_resize(table, lens + 1, c["pages"], c["page"])
        return [table, src, dst] + state
    table, src, dst, count = A.pages_compact(s["table"], c["pages"])
    A.cache_copy_pages(cache, src, dst)
    return [table, src, dst, count] + state


# ------------------------------------------------------------------ from the definitions

def _nearest(x, bits):
    """x (float64) to `bits` significant bits, halves to even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(torch.ldexp(m, torch.tensor(bits, device=DEV))), e - bits)


def _exact_pages(case, s):
    """The new table, pairs and (compact) count, one entry at a time."""
    table, page, pages = s["table"].cpu().numpy(), case.get("page"), case["pages"]
    if case["op"] == "compact":
        used = sorted(set(table[table >= 0].tolist()))
        inside = set(used)
        src = [p for p in used if p >= len(used)]
        dst = [p for p in range(len(used)) if p not in inside]
        to = dict(zip(src, dst))
        new = np.array([[to.get(p, p) for p in row] for row in table.tolist()], np.int32)
        room = min(pages // 2, table.size)
        pad = [-1] * (room - len(src))
        return new, np.array(src + pad, np.int32), np.array(dst + pad, np.int32), np.array([len(used)], np.int32)
    lens, parents = s["lens"].cpu().numpy(), s["parents"].cpu().numpy()
    new, full, owner = [], set(), {}
    for i, a in enumerate(parents.tolist()):
        n = int(lens[a])
        row = table[a, :-(-n // page)].tolist()
        full.update(row[:n // page])
        if n % page:
            owner.setdefault(row[-1], i)
        new.append((row, n))
    want = [i for i, (row, n) in enumerate(new) if n % page and (owner[row[-1]] != i or row[-1] in full)]
    named = {p for i, (row, _) in enumerate(new) for p in (row[:-1] if i in set(want) else row)}
    free = (p for p in range(pages) if p not in named)
    src, dst = np.full(len(new), -1, np.int32), np.full(len(new), -1, np.int32)
    for i in want:
        src[i], dst[i] = new[i][0][-1], next(free)
        new[i][0][-1] = int(dst[i])
    out = np.full(table.shape, -1, np.int32)
    named = {p for row, _ in new for p in row}
    free = (p for p in range(pages) if p not in named)
    for i, (row, n) in enumerate(new):
        row += [next(free) for _ in range(-(-(n + 1) // page) - len(row))]
        out[i, :len(row)] = row
    return out, src, dst


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("adapters", "gradients"):
        x, down, up = s["x"].double(), s["down"].double(), s["up"].double()
        scale, index = s["scale"].double(), s["index"]
        if op == "adapters":
            out = s["y"].double()
            for i in range(case["adapters"]):
                at = torch.nonzero(index == i)[:, 0]
                out[at] += scale[i] * ((x[at] @ down[i].T) @ up[i])
            return out
        dy, dx, ddown, dup = s["dy"].double(), s["dx"].double(), torch.zeros_like(down), torch.zeros_like(up)
        for i in range(case["adapters"]):
            at = torch.nonzero(index == i)[:, 0]
            e = scale[i] * (dy[at] @ up[i].T)
            dx[at] += e @ down[i]
            ddown[i] = e.T @ x[at]
            dup[i] = scale[i] * ((x[at] @ down[i].T).T @ dy[at])
        return {"dx": dx, "down": ddown, "up": dup}
    if op == "linear":
        n, k = case["n"], case["k"]
        g = (torch.arange(16, dtype=torch.float64, device=DEV) / 15.0) ** (1.0 / float(np.float32(ALPHA)))
        w = torch.empty((n, k), dtype=torch.float64, device=DEV)
        for i in range(8):
            w[:, i::8] = g[torch.remainder(torch.div(s["packed"].long(), 16 ** i, rounding_mode="floor"), 16)]
        w *= torch.repeat_interleave(s["scale"].double().view(n, -1), case["group"] or k, 1)
        w = _nearest(w, 8)
        for i in range(32):
            w[:, i::32] *= 1.0 - 2.0 * torch.remainder(torch.div(s["sign"].long(), 2 ** i, rounding_mode="floor"), 2).double()
        return s["dy"].double() @ w
    if op == "verify":
        t, counts, paths, drawn = case["draft"], [], [], []
        tokens, u = s["tokens"].cpu().numpy(), s["uniforms"].double().cpu().numpy()
        for b in range(case["batch"]):
            parents = s["parents"][b].cpu().numpy() if case["tree"] else np.arange(-1, t - 1)
            path, refused, left = [0], [], 1.0
            for i in range(1, t):
                if parents[i] != path[-1]:
                    continue
                px = float(s["p"][b, path[-1], int(tokens[b, i])])
                if case["tree"]:
                    px = 0.0 if any(tokens[b, j] == tokens[b, i] for j in refused) else px
                    ok = u[b, i] * left < px
                else:
                    ok = u[b, i] * float(s["q"][b, i - 1, int(tokens[b, i])]) < px
                if ok:
                    path, refused, left = path + [i], [], 1.0
                else:
                    refused, left = refused + [i], left - px
            w = s["p"][b, path[-1]].double()
            if refused and not case["tree"]:
                w = torch.relu(w - s["q"][b, refused[0] - 1].double())
            elif refused:
                w[torch.from_numpy(tokens[b, refused].astype(np.int64)).to(DEV)] = 0.0
            cum = np.cumsum(w.cpu().numpy())
            drawn.append(int(np.nonzero(cum > u[b, 0] * cum[-1])[0][0]))
            counts.append(len(path))
            paths.append(path + [-1] * (t - len(path)))
        return {"kept": torch.tensor(paths, dtype=torch.int32, device=DEV),
                "count": torch.tensor(counts, dtype=torch.int32, device=DEV),
                "next": torch.tensor(drawn, dtype=torch.int32, device=DEV)}
    found = _exact_pages(case, s)
    state = []
    for side in s["sides"]:
        for t in side.values():
            if t is not None:
                for a, b in zip(found[1].tolist(), found[2].tolist()):
                    if b >= 0:
                        t[b].copy_(t[a])
                state.append(t)
    return [torch.from_numpy(f).to(DEV) for f in found] + state
