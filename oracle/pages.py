"""The page operations of a cache, one request after another, on numpy state changed in place.

table [S, pages_per_seq], lens [S], refs [num_pages]; pools: arrays with the page first.
"""
from __future__ import annotations

import numpy as np


def _need(n, page_size):
    return -(-int(n) // page_size)


def free_list(refs):
    return [int(p) for p in np.flatnonzero(refs == 0)]


def extend(table, lens, refs, page_size, slots, add):
    """False (and nothing changed) if the request cannot be met."""
    slots = [int(s) for s in slots]
    if len(set(slots)) < len(slots) or any(s < 0 or s >= len(lens) for s in slots):
        return False
    if any(a < 0 or int(lens[s]) + int(a) > table.shape[1] * page_size for s, a in zip(slots, add)):
        return False
    free = free_list(refs)
    if sum(_need(lens[s] + a, page_size) - _need(lens[s], page_size) for s, a in zip(slots, add)) > len(free):
        return False
    for s, a in zip(slots, add):
        for c in range(_need(lens[s], page_size), _need(lens[s] + a, page_size)):
            table[s, c] = free.pop(0)
            refs[table[s, c]] = 1
        lens[s] += a
    return True


def fork(table, lens, refs, page_size, src, dst, pools):
    src, dst = [int(s) for s in src], [int(s) for s in dst]
    if any(s < 0 or s >= len(lens) for s in src + dst) or len(set(dst)) < len(dst) or set(src) & set(dst) or any(lens[d] for d in dst):
        return False
    free = free_list(refs)
    if sum(lens[s] % page_size > 0 for s in src) > len(free):
        return False
    for s, d in zip(src, dst):
        full = int(lens[s]) // page_size
        table[d, :full] = table[s, :full]
        for p in table[s, :full]:
            refs[p] += 1
        if lens[s] % page_size:
            new = free.pop(0)
            table[d, full] = new
            refs[new] = 1
            for x in pools:
                x[new] = x[table[s, full]]
        lens[d] = lens[s]
    return True


def free(table, lens, refs, page_size, slots):
    for s in slots:
        for c in range(_need(lens[s], page_size)):
            refs[table[s, c]] -= 1
            table[s, c] = -1
        lens[s] = 0


def compact(table, lens, refs, page_size, pools):
    """(table, refs, remap, n_live) of the new places; the pools are changed in place."""
    n_live = int((refs > 0).sum())
    movers = [p for p in range(len(refs)) if refs[p] > 0 and p >= n_live]
    holes = [p for p in range(n_live) if refs[p] <= 0]
    remap = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    new_refs = refs.copy()
    for a, z in zip(movers, holes):
        remap[a] = z
        new_refs[z], new_refs[a] = refs[a], 0
        for x in pools:
            x[z] = x[a]
    new_table = table.copy()
    for s in range(len(lens)):
        for c in range(_need(lens[s], page_size)):
            new_table[s, c] = remap[table[s, c]]
    return new_table, new_refs, remap, n_live
