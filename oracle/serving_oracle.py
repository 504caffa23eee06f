"""Plain oracle of what a server with many requests does between its layers: pages of a cache
forked, taken, freed and drawn together, and drafted tokens verified.  Written from the
definitions in include/opq_attention.h, one entry and one token at a time, in Python's
integers and float64 (test infrastructure: it shares nothing with the kernels)."""
import math

import numpy as np


def _named(table, pages):
    return {int(e) for e in np.asarray(table).ravel() if 0 <= e < pages}


def _free(named, pages):
    return [p for p in range(pages) if p not in named]


def resize(table, lens, pages, page):
    """(table, missing)"""
    table = np.array(table, np.int64)
    rows, columns = table.shape
    out = np.full((rows, columns), -1, np.int64)
    lacking = []
    for i in range(rows):
        need = -(-min(max(int(lens[i]), 0), columns * page) // page)
        for c in range(need):
            if 0 <= table[i, c] < pages:
                out[i, c] = table[i, c]
            else:
                lacking.append((i, c))
    free = _free(_named(out, pages), pages)
    for (i, c), p in zip(lacking, free):
        out[i, c] = p
    return out.astype(np.int32), max(0, len(lacking) - len(free))


def fork(table, lens, parents, pages, page):
    """(table, lens, src, dst, missing)"""
    table = np.array(table, np.int64)
    rows, columns = table.shape
    new = np.full((len(parents), columns), -1, np.int64)
    new_lens = np.zeros(len(parents), np.int64)
    full, owner = set(), {}
    ends = [None] * len(parents)
    for i, a in enumerate(parents):
        if not 0 <= a < rows:
            continue
        n = min(max(int(lens[a]), 0), columns * page)
        new_lens[i] = n
        for c in range(-(-n // page)):
            e = int(table[a, c])
            new[i, c] = e if 0 <= e < pages else -1
            if new[i, c] < 0:
                continue
            if (c + 1) * page <= n:
                full.add(e)
            else:
                ends[i] = c
                owner.setdefault(e, i)
    src, dst = np.full(len(parents), -1, np.int64), np.full(len(parents), -1, np.int64)
    copies = [i for i, c in enumerate(ends) if c is not None and (int(new[i, c]) in full or owner[int(new[i, c])] != i)]
    old = {i: int(new[i, ends[i]]) for i in copies}
    free = _free(full | set(owner), pages)
    for k, i in enumerate(copies):
        new[i, ends[i]] = -1
        if k < len(free):
            new[i, ends[i]], src[i], dst[i] = free[k], old[i], free[k]
    out = [a.astype(np.int32) for a in (new, new_lens, src, dst)]
    return out[0], out[1], out[2], out[3], max(0, len(copies) - len(free))


def compact(table, pages):
    """(table, src, dst, used), src and dst without padding"""
    used = sorted(_named(table, pages))
    src = [p for p in used if p >= len(used)]
    dst = [p for p in range(len(used)) if p not in set(used)]
    to = dict(zip(src, dst))
    new = [[to.get(int(e), int(e)) if 0 <= e < pages else -1 for e in row] for row in np.asarray(table)]
    return np.array(new, np.int32).reshape(np.shape(table)), src, dst, len(used)


def _proper(v):
    v = float(v)
    return v if 0.0 < v < math.inf else 0.0


def verify(p, tokens, u, q=None, parents=None, count=None):
    """(kept, number, next, weights) of one sequence: p [draft][vocab], q [draft-1][vocab]; weights
    are those that next is drawn from."""
    draft, vocab = len(tokens), len(p[0])
    count = draft if count is None else min(max(int(count), 0), draft)
    if count == 0:
        return [-1] * draft, 0, -1, None
    parents = list(range(-1, draft - 1)) if parents is None else parents
    path, tested, left = [0], [], 1.0
    while True:
        node, after = path[-1], None
        tested, left = [], 1.0
        for t in range(node + 1, count):
            if parents[t] != node:
                continue
            x = int(tokens[t])
            px = _proper(p[node][x]) if 0 <= x < vocab else 0.0
            if q is None:
                if x in tested:
                    px = 0.0
                keep = px > 0.0 and float(u[t]) * left < px
            else:
                qx = _proper(q[t - 1][x]) if 0 <= x < vocab else 0.0
                keep = px > 0.0 and float(u[t]) * qx < px
            if keep:
                after = t
                break
            tested.append(x)
            left -= px
        if after is None:
            break
        path.append(after)
    w = [_proper(v) for v in p[path[-1]]]
    if tested and q is not None:
        w = [max(a - _proper(b), 0.0) for a, b in zip(w, q[path[-1]])]
    elif tested:
        w = [0.0 if i in set(tested) else a for i, a in enumerate(w)]
    return path + [-1] * (draft - len(path)), len(path), draw(w, float(u[0])), w


def draw(w, u):
    total = math.fsum(w)
    last = max((i for i, v in enumerate(w) if v > 0.0), default=-1)
    at = 0.0
    for i, v in enumerate(w):
        at += v
        if v > 0.0 and at > u * total:
            return i
    return last
