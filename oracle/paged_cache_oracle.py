"""Plain CPU oracle of the paged key/value cache operators (TEST INFRASTRUCTURE ONLY).

numpy in float64, one sequence, node and head at a time; pages are looked up entry by entry.
Nothing of the product path is used here.  The functions that move rows or count pages change
the arrays they are given, as the operators do.
"""

from __future__ import annotations

import numpy as np

__all__ = ["positions", "tree_attention", "append", "commit", "resize", "fork"]


def positions(table_row, page_size, pages, first, last, books=None):
    """[(position, page, slot)] of positions first <= x < last that have a page.  `books`: (entries
    that the sequence holds, counts of all pages); a page named behind those that somebody holds is
    another sequence's."""
    cap = len(table_row) * page_size
    out = []
    for x in range(first, min(last, cap)):
        page = int(table_row[x // page_size])
        if not 0 <= page < pages:
            continue
        if books is not None and x // page_size >= books[0] and books[1][page] != 0:
            continue
        out.append((x, page, x % page_size))
    return out


def _books(held, refcount, b):
    return None if held is None or refcount is None else (int(held[b]), refcount)


def _length(lens, b, cap):
    return min(max(int(lens[b]), 0), cap)


def tree_attention(q, k, v, table, lens, mask=None, nodes=None, scale=None, held=None,
                   refcount=None):
    """q [B, N, Hq, D], k, v [pages, page_size, Hkv, D] (one layer) in float64.

    Returns out [B, N, Hq, D], lse [B, N, Hq] and what error bounds are made of: absolute
    [B, N, Hq, D] = sum of weight * |v|, reach [B, N, Hq] = max over seen keys of
    scale * sum |q k|, and count [B, N] = keys seen."""
    B, N, Hq, D = q.shape
    pages, page_size, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    cap = table.shape[1] * page_size
    out = np.zeros((B, N, Hq, D))
    absolute = np.zeros((B, N, Hq, D))
    lse = np.full((B, N, Hq), -np.inf)
    reach = np.zeros((B, N, Hq))
    count = np.zeros((B, N), dtype=np.int64)
    for b in range(B):
        length = _length(lens, b, cap)
        n = N if nodes is None else min(max(int(nodes[b]), 0), N)
        rows = positions(table[b], page_size, pages, 0, length + n, _books(held, refcount, b))
        for i in range(n):
            seen = [(p, s) for x, p, s in rows
                    if x < length or (x - length <= i if mask is None
                                      else mask[b, i, x - length] != 0)]
            count[b, i] = len(seen)
            if not seen:
                continue
            p = np.array([x[0] for x in seen])
            s = np.array([x[1] for x in seen])
            for h in range(Hq):
                kk, vv = k[p, s, h // G], v[p, s, h // G]
                with np.errstate(invalid="ignore", over="ignore"):
                    z = scale * (kk @ q[b, i, h])
                    m = z.max()
                    w = np.exp(z - m)
                    total = w.sum()
                    out[b, i, h] = (w @ vv) / total
                    lse[b, i, h] = m + np.log(total)
                    absolute[b, i, h] = (w @ np.abs(vv)) / total
                    reach[b, i, h] = scale * (np.abs(kk) @ np.abs(q[b, i, h])).max()
    return dict(out=out, lse=lse, absolute=absolute, reach=reach, count=count)


def append(k, v, k_new, v_new, table, lens, nodes=None, held=None, refcount=None):
    """Writes k_new, v_new [B, N, Hkv, D] behind the committed tokens of one layer's k, v."""
    pages, page_size = k.shape[:2]
    B, N = k_new.shape[:2]
    for b in range(B):
        length = _length(lens, b, table.shape[1] * page_size)
        n = N if nodes is None else min(max(int(nodes[b]), 0), N)
        for x, page, slot in positions(table[b], page_size, pages, length, length + n,
                                       _books(held, refcount, b)):
            k[page, slot] = k_new[b, x - length]
            v[page, slot] = v_new[b, x - length]


def commit(k, v, table, lens, last, parent=None, N=None, held=None, refcount=None):
    """Moves the accepted path's rows of k, v [layers, pages, page_size, Hkv, D] together;
    returns the new lengths."""
    pages, page_size = k.shape[1:3]
    cap = table.shape[1] * page_size
    N = parent.shape[1] if parent is not None else N
    out = np.zeros(len(lens), dtype=np.int32)
    for b in range(len(lens)):
        length = _length(lens, b, cap)
        out[b] = length
        node = int(last[b])
        if not 0 <= node < N:
            continue
        path = [node]
        while path[0] != 0:
            up = path[0] - 1 if parent is None else int(parent[b, path[0]])
            if not 0 <= up < path[0]:
                path = None
                break
            path.insert(0, up)
        if path is None:
            continue
        where = [positions(table[b], page_size, pages, length + x, length + x + 1,
                           _books(held, refcount, b))
                 for x in path + list(range(len(path)))]
        if not all(where):
            continue
        src, dst = where[:len(path)], where[len(path):]
        rows = [(k[:, s[0][1], s[0][2]].copy(), v[:, s[0][1], s[0][2]].copy()) for s in src]
        for d, (a, c) in zip(dst, rows):
            k[:, d[0][1], d[0][2]] = a
            v[:, d[0][1], d[0][2]] = c
        out[b] = length + len(path)
    return out


def resize(table, lens, held, refcount, want, page_size, new_lens=None):
    """Pages given back, then taken, lowest index first; returns ok.  New lengths that cut into
    pages which stay and are shared are out of range.  The entries that a refused sequence asked
    for are cleared."""
    S, width = table.shape
    ok = np.zeros(S, dtype=np.int32)
    need = np.zeros(S, dtype=np.int64)
    before = refcount.copy()
    for b in range(S):
        good = 0 <= held[b] <= width
        if good and new_lens is not None:
            good = 0 <= new_lens[b] <= int(held[b]) * page_size
            old = min(max(int(lens[b]), 0), int(held[b]) * page_size)
            if good and new_lens[b] < old and want[b] != 0:
                # entries that stay: all of them, unless the wish is one that will be followed
                stay = held[b]
                if new_lens[b] <= want[b] <= width * page_size:
                    stay = -(-int(want[b]) // page_size)
                for j in range(new_lens[b] // page_size, min(-(-old // page_size), stay)):
                    good = good and not (0 <= table[b, j] < len(before) and before[table[b, j]] > 1)
            if good:
                lens[b] = new_lens[b]
        good = good and (want[b] <= 0 or lens[b] <= want[b] <= width * page_size)
        ok[b] = good
        if not good and held[b] >= 0 and want[b] > 0:
            table[b, held[b]:-(-min(int(want[b]), width * page_size) // page_size)] = -1
        need[b] = held[b] if not good or want[b] < 0 else -(-int(want[b]) // page_size)
        for j in range(need[b], held[b]):
            if 0 <= table[b, j] < len(refcount):
                refcount[table[b, j]] -= 1
    free = [p for p in range(len(refcount)) if refcount[p] == 0]
    full = False
    for b in range(S):
        if not ok[b]:
            continue
        grow = need[b] - held[b]
        if grow > 0:
            full = full or grow > len(free)
            if full:
                ok[b] = 0
                table[b, held[b]:need[b]] = -1
                continue
            for j in range(held[b], need[b]):
                table[b, j] = free.pop(0)
                refcount[table[b, j]] = 1
        held[b] = need[b]
        if want[b] == 0:
            lens[b] = 0
    return ok


def fork(k, v, table, lens, held, refcount, src, dst):
    """Sequences src continued as dst; k, v [layers, pages, page_size, Hkv, D] or None; returns
    ok."""
    S, width = table.shape
    page_size = k.shape[2]
    ok = np.zeros(len(src), dtype=np.int32)
    taken = set()
    good = []
    for f, (x, d) in enumerate(zip(src, dst)):
        first = d not in taken
        taken.add(d)
        if not (0 <= x < S and 0 <= d < S) or not first or d in src or held[d] != 0:
            continue
        if lens[x] < 0 or not 0 <= held[x] <= width or lens[x] > held[x] * page_size:
            continue
        full, rest = divmod(int(lens[x]), page_size)
        if rest and not 0 <= table[x, full] < len(refcount):
            continue
        good.append((f, x, d, full, rest))
    free = [p for p in range(len(refcount)) if refcount[p] == 0]
    for f, x, d, full, rest in good:
        if rest:
            if not free:
                continue
            page = free.pop(0)
            refcount[page] = 1
            old = table[x, full]
            table[d, full] = page
            k[:, page, :rest] = k[:, old, :rest]
            v[:, page, :rest] = v[:, old, :rest]
        for j in range(full):
            table[d, j] = table[x, j]
            if 0 <= table[x, j] < len(refcount):
                refcount[table[x, j]] += 1
        held[d] = full + (1 if rest else 0)
        lens[d] = lens[x]
        ok[f] = 1
    return ok
