"""Plain restatement of the paged key-value cache operators: attention in fp64, one query row and
head at a time, and the upkeep of the pages on Python lists, one sequence after the other.  Shares
nothing with the CUDA path.  Contracts: include/misa.h ("Paged key-value cache")."""

from __future__ import annotations

import numpy as np


def attention_row(q, k, v, table, page_size, seen, scale):
    """One query row.  q [Hq, d]; k, v [num_pages, page_size, Hkv, d]; table: the sequence's
    pages; seen: token ids.  Returns out [Hq, d], lse [Hq] and, per head, the weighted mean of
    |v| [Hq, d] (the scale of an output's rounding errors) and the largest scale * sum |q k|."""
    Hq, d = q.shape
    Hkv = k.shape[2]
    out, mean_abs = np.zeros((Hq, d)), np.zeros((Hq, d))
    lse, mag = np.full(Hq, -np.inf), np.zeros(Hq)
    if len(seen) == 0:
        return out, lse, mean_abs, mag
    pages = np.array([table[s // page_size] for s in seen])
    offs = np.array([s % page_size for s in seen])
    for j in range(Hq):
        kk, vv = k[pages, offs, j // (Hq // Hkv)], v[pages, offs, j // (Hq // Hkv)]
        z = scale * (kk @ q[j])
        m = z.max()
        if m == -np.inf:
            continue
        p = np.exp(z - m)
        out[j] = (p @ vv) / p.sum()
        mean_abs[j] = (p @ np.abs(vv)) / p.sum()
        lse[j] = m + np.log(p.sum())
        mag[j] = abs(scale) * (np.abs(kk) @ np.abs(q[j])).max()
    return out, lse, mean_abs, mag


class OutOfPages(Exception):
    pass


def resize(table, refs, old, new, page_size):
    """table: list of rows; refs: list.  Returns (table, refs, copies): copies are (from, to)
    pages whose contents follow."""
    table, before, refs = [list(r) for r in table], list(refs), list(refs)
    free = [p for p, r in enumerate(before) if r == 0]
    left, copies, cap = list(before), [], len(table[0]) * page_size

    def take():
        if not free:
            raise OutOfPages
        p = free.pop(0)
        refs[p] = 1
        return p

    for n, row in enumerate(table):
        o, x = old[n], new[n]
        if not (0 <= o <= cap and 0 <= x <= cap):
            continue
        oldp, newp = -(-o // page_size), -(-x // page_size)
        if x > o and o % page_size:
            p = row[o // page_size]
            if left[p] > 1:          # others hold it: this sequence takes a copy
                left[p] -= 1
                refs[p] -= 1
                row[o // page_size] = take()
                copies.append((p, row[o // page_size]))
        for c in range(oldp, newp):
            row[c] = take()
        for c in range(newp, oldp):
            refs[row[c]] -= 1
        for c in range(newp, len(row)):
            row[c] = -1
    return table, refs, copies


def fork(table, refs, parent):
    out = []
    for n, p in enumerate(parent):
        if p == -1:
            out.append([-1] * len(table[n]))
        elif 0 <= p < len(table):
            out.append(list(table[p]))
        else:
            out.append(list(table[n]))
    refs = list(refs)
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] -= 1
    for row in out:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return out, refs


def compact(table, refs):
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] == 0]
    copies = list(zip([p for p in live if p >= n], holes))
    to, refs = dict(copies), list(refs)
    for a, b in copies:
        refs[b], refs[a] = refs[a], 0
    return [[to.get(e, e) for e in row] for row in table], refs, n, copies
