"""Oracle of the page operators (plain Python, request by request).

Tables are lists of rows, lengths and counts lists of ints; copies come back
as (from, to, cells) and are applied by the caller. No code is shared with the
CUDA path.
"""

from __future__ import annotations


def pages_of(n: int, bs: int) -> int:
    return -(-n // bs)


def fork(table, lens, refs, parents, bs):
    """(table, lens, refs) of the batch that continues ``parents``."""
    width = len(table[0]) if table else 0
    refs = list(refs)
    for r, row in enumerate(table):
        children = sum(p == r for p in parents)
        for page in row[:pages_of(lens[r], bs)]:
            refs[page] += children - 1
    return ([list(table[p]) if p >= 0 else [-1] * width for p in parents], [lens[p] if p >= 0 else 0 for p in parents], refs)


def resize(table, lens, new, refs, bs):
    """(table, lens, refs, copies, refused)."""
    free = [p for p, r in enumerate(refs) if r <= 0]
    table, out, now = [list(r) for r in table], list(lens), list(refs)

    def shared_last(r):
        n = lens[r]
        if new[r] <= n or n % bs == 0:
            return None
        page = table0[r][n // bs]
        return page if refs[page] > 1 else None

    table0 = [list(r) for r in table]
    wants = [shared_last(r) for r in range(len(table))]
    taken, copies, refused = 0, [], []
    for r, row in enumerate(table):
        have, want = pages_of(lens[r], bs), pages_of(new[r], bs)
        page = wants[r]
        sharers = [k for k, p in enumerate(wants) if p == page] if page is not None else []
        keeps = page is not None and len(sharers) == refs[page] and sharers[-1] == r
        copy = page is not None and not keeps
        need = int(copy) + max(0, want - have)
        first = taken
        taken += need
        if (need or keeps) and taken > len(free):
            refused.append(r)
            continue
        got = free[first:taken]
        out[r] = new[r]
        if copy:
            copies.append((page, got[0], lens[r] % bs))
            row[have - 1] = got[0]
            now[page] -= 1
            got = got[1:]
        for i, p in enumerate(got):
            row[have + i] = p
        for i in range(want, have):
            now[row[i]] -= 1
            row[i] = -1
        for p in free[first:taken]:
            now[p] = 1
    return table, out, now, copies, refused


def compact(table, lens, refs, bs):
    """(table, refs, moves, copies)."""
    held = [p for p, r in enumerate(refs) if r > 0]
    top = len(held)
    movers = [p for p in held if p >= top]
    holes = [p for p in range(top) if refs[p] <= 0]
    moves = [p if refs[p] > 0 else -1 for p in range(len(refs))]
    out = list(refs)
    for a, b in zip(movers, holes):
        moves[a], out[b], out[a] = b, refs[a], 0
    table = [[moves[p] if i < pages_of(n, bs) else p for i, p in enumerate(row)] for row, n in zip(table, lens)]
    return table, out, moves, list(zip(movers, holes))
