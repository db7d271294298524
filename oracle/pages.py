"""The page operators on lists, one entry after the other.

Test infrastructure, written from the definitions in include/indexer_pages.h,
sharing no code with the HIP path.  A pool is refs (a list), table (a list of
rows), lens (a list) and caches (NumPy arrays [n_pages, ...]); every function
changes them in place.
"""
from __future__ import annotations


def copy(caches, source, target):
    n = len(caches[0])
    old = [c.copy() for c in caches]
    for a, b in zip(source, target):
        if 0 <= a < n and 0 <= b < n and a != b:
            for c, o in zip(caches, old):
                c[b] = o[a]


def _first(rows, n_rows):
    """Which entries of a list count."""
    named = set()
    out = []
    for r in rows:
        out.append(0 <= r < n_rows and r not in named)
        named.add(r)
    return out


def _length(lens, row, cols, bs):
    return min(max(lens[row], 0), cols * bs)


def fork(caches, refs, table, lens, parents, children, bs):
    rows, cols = len(table), len(table[0]) if table else 0
    free = [p for p, r in enumerate(refs) if r <= 0]
    fresh = []
    for p, c, ok in zip(parents, children, _first_pairs(parents, children, rows)):
        if not ok:
            fresh.append(-3)
            continue
        length = _length(lens, p, cols, bs)
        full, rest = divmod(length, bs)
        if rest and not free:
            table[c], lens[c] = [-1] * cols, 0
            fresh.append(-2)
            continue
        row = [e if 0 <= e < len(refs) else -1 for e in table[p][:full]]
        for e in row:
            if e >= 0:
                refs[e] += 1
        row += [-1] * (cols - full)
        page = -1
        if rest:
            turn = free.pop(0)
            if 0 <= table[p][full] < len(refs):
                page = row[full] = turn
                refs[page] = 1
                for a in caches:
                    a[page] = a[table[p][full]]
        table[c], lens[c] = row, length
        fresh.append(page)
    return fresh


def _first_pairs(parents, children, n_rows):
    """A child's first mention decides, whether its parent is there or not."""
    return [ok and 0 <= p < n_rows and p != c for p, c, ok in zip(parents, children, _first(children, n_rows))]


def grow(refs, table, lens, rows, tokens, bs, new_tokens=None):
    n_rows, cols = len(table), len(table[0]) if table else 0
    free = [p for p, r in enumerate(refs) if r <= 0]
    asked, slots = 0, []
    for i, (r, ok) in enumerate(zip(rows, _first(rows, n_rows))):
        new = tokens if new_tokens is None else min(max(new_tokens[i], 0), tokens)
        mine = [-1] * tokens
        slots.append(mine)
        if not ok:
            continue
        length = _length(lens, r, cols, bs)
        held, want = -(-length // bs), -(-(length + new) // bs)
        if want > cols:
            continue
        if new and length % bs and not 0 <= table[r][length // bs] < len(refs):
            continue
        asked += want - held
        if want > held and asked > len(free):
            continue
        for k in range(held, want):
            page = free[asked - want + k]
            table[r][k] = page
            refs[page] = 1
        for k in range(new):
            page = table[r][(length + k) // bs]
            mine[k] = page * bs + (length + k) % bs
        lens[r] = length + new
    return slots


def free(refs, table, lens, rows):
    for r, ok in zip(rows, _first(rows, len(table))):
        if not ok:
            continue
        for e in table[r]:
            if 0 <= e < len(refs):
                refs[e] -= 1
        table[r], lens[r] = [-1] * len(table[r]), 0


def compact(caches, refs, table):
    n = len(refs)
    live = sum(r > 0 for r in refs)
    holes = [p for p in range(live) if refs[p] <= 0]
    late = [p for p in range(live, n) if refs[p] > 0]
    place = [p if r > 0 else -1 for p, r in enumerate(refs)]
    for a, b in zip(late, holes):
        place[a] = b
        refs[b], refs[a] = refs[a], 0
        for c in caches:
            c[b] = c[a]
    for row in table:
        row[:] = [place[e] if 0 <= e < n else -1 for e in row]
    return place, live
