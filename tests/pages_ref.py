"""The pages' bookkeeping in plain Python, entry by entry: what the calls do
to refs, tables and lists, and what a list's moves do to a pool."""
from __future__ import annotations


def fork(refs, P, src_table, src_lens, parents, stride):
    table, lens = [], []
    for p in parents:
        n = 0 if p < 0 else src_lens[p]
        row = [src_table[p][j] if j * P < n else -1 for j in range(stride)]
        for e in row:
            if e >= 0:
                refs[e] += 1
        table.append(row)
        lens.append(n)
    return table, lens


def free(refs, table, first=None, end=None):
    for s, row in enumerate(table):
        for j in range(first[s] if first else 0, end[s] if end else len(row)):
            if row[j] >= 0:
                refs[row[j]] -= 1
                row[j] = -1


def free_window(refs, P, table, lens, window, sinks):
    for row, n in zip(table, lens):
        for j, e in enumerate(row):
            unseen = all(sinks <= x <= n - window for x in range(j * P, (j + 1) * P))
            if e >= 0 and unseen:
                refs[e] -= 1
                row[j] = -1


def grow(refs, P, table, lens, rows):
    """Returns the moves [(src, dst, positions)], or None when pages run out (nothing changes)."""
    wants = []
    for s, n in enumerate(lens):
        if n == 0:
            continue
        for j in range((n - rows) // P, (n - 1) // P + 1):
            e = table[s][j]
            if e < 0:
                wants.append((s, j, -1, 0))
            elif refs[e] > 1:
                wants.append((s, j, e, max(0, n - rows - j * P)))
    free_ids = [i for i, r in enumerate(refs) if r == 0]
    if len(free_ids) < len(wants):
        return None
    moves = []
    for (s, j, e, n), page in zip(wants, free_ids):
        table[s][j] = page
        moves.append((e, page, n))
    for (_, _, e, _), page in zip(wants, free_ids):
        refs[page] = 1
        if e >= 0:
            refs[e] -= 1
    return moves


def compact(refs, table):
    n_live = sum(r > 0 for r in refs)
    src = [i for i, r in enumerate(refs) if r > 0 and i >= n_live]
    dst = [i for i, r in enumerate(refs) if r == 0 and i < n_live]
    to = dict(zip(src, dst))
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    for row in table:
        row[:] = [to.get(e, e) for e in row]
    return list(zip(src, dst)), n_live


def move(pool, moves):
    """pool: a tensor [n_pages][Hkv][P][d], changed in place."""
    for src, dst, n in moves:
        if src >= 0 and n > 0:
            pool[dst, :, :n] = pool[src, :, :n].clone()
