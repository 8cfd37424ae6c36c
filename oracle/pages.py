"""The upkeep of a paged KV cache, step by step in plain Python — test infrastructure only.

Caches are lists of arrays [layers, pages, page_size, ...] (K, V and scales alike); tables, lengths and
counts are plain lists.  Nothing here is computed, so results are exact.
"""
from __future__ import annotations


def accept(caches, base, path, rows_of):
    """Sequence by sequence: the rows of drafts path[b][j] become those of slots base[b] + j, all read before any
    is written.  rows_of(b, slot) -> index of the slot within a layer."""
    for x in caches:
        for b, steps in enumerate(path):
            got = [x[(slice(None),) + rows_of(b, base[b] + d)].copy() for d in steps]
            for j, row in enumerate(got):
                x[(slice(None),) + rows_of(b, base[b] + j)] = row


def copy_pages(caches, src, dst):
    for x in caches:
        x[:, dst] = x[:, src].copy()


def fork(caches, table, lens, refs, parents, keep, new, page, max_pages):
    """Returns (table, lens, refs, free pages left) of the children; None in place of the table when the pages
    are too few (the caches are then untouched)."""
    N = len(refs)
    refs = list(refs)
    for row, n in zip(table, lens):
        for p in row[:-(-n // page)]:
            refs[p] -= 1
    kept = []
    for a, k, n in zip(parents, keep, new):
        k = max(0, min(k, n, lens[a])) if a >= 0 else 0
        kept.append(k)
        for p in (table[a][:k // page] if a >= 0 else []):
            refs[p] += 1
    rows, cut = [], []
    shared = [r > 0 for r in refs]  # held whole by somebody, or pinned
    for c, (a, k) in enumerate(zip(parents, kept)):
        rows.append(list(table[a][:k // page]) if a >= 0 else [])
        if k % page:
            p = table[a][k // page]
            if not shared[p] and refs[p] == 0:
                refs[p] = 1
                rows[c].append(p)
            else:
                cut.append((c, p, k % page))
    need = [-(-n // page) - len(r) for n, r in zip(new, rows)]
    free = [p for p in range(N) if refs[p] == 0]
    if sum(need) > len(free):
        return None, None, None, len(free) - sum(need)
    for c, n in enumerate(need):
        for _ in range(n):
            p = free.pop(0)
            refs[p] = 1
            rows[c].append(p)
    for c, p, n in cut:
        for x in caches:
            x[:, rows[c][kept[c] // page], :n] = x[:, p, :n]
    return [r + [-1] * (max_pages - len(r)) for r in rows], list(new), refs, len(free)


def compact(caches, table, refs):
    """Returns (table, refs, page_map, live pages, pages moved)."""
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    slots = [p for p in range(n) if refs[p] <= 0]
    to = {p: (p if p < n else None) for p in live}
    for p in live:
        if p >= n:
            q = to[p] = slots.pop(0)
            for x in caches:
                x[:, q] = x[:, p]
    page_map = [to.get(p, -1) for p in range(len(refs))]
    out = [0] * len(refs)
    for p in live:
        out[to[p]] = refs[p]
    return [[page_map[p] if p >= 0 else -1 for p in row] for row in table], out, page_map, n, sum(p >= n for p in live)
