"""Pages that sequences share: counts, forks, growth, freeing and compaction,
one sequence after the other.

TEST INFRASTRUCTURE ONLY (see the package docstring): it shares no code with
the CUDA library.  ``planes`` is a list of arrays whose first index is the page.
"""

from __future__ import annotations

import numpy as np


def held(n, page):
    return -(-int(n) // page)


def fork(refs, table, kv_len, page, parent, child):
    """Returns whether every fork was taken."""
    parent, child = [int(x) for x in parent], [int(x) for x in child]
    fine = True
    start = kv_len.copy()
    for p, c in zip(parent, child):
        rows = range(len(kv_len))
        if p not in rows or c not in rows or child.count(c) > 1 or c in parent or start[c] != 0:
            fine = False
            continue
        for i in range(held(start[p], page)):
            table[c, i] = table[p, i]
            refs[table[p, i]] += 1
        kv_len[c] = start[p]
    return fine


def extend(refs, table, planes, page, old, new):
    """Returns whether there were pages enough; if not, nothing changes but entries
    to be filled (-1) and the new lengths of those that lack room (-1)."""
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    r, t, copies, fills = refs.copy(), table.copy(), [], []
    for b in range(len(old)):
        at, last = int(old[b]) // page, held(new[b], page)
        if new[b] > old[b] and old[b] % page and r[t[b, at]] >= 2:
            copies.append((b, at, int(t[b, at])))
            r[t[b, at]] -= 1
            fills.append((b, at))
        fills += [(b, i) for i in range(held(old[b], page), last)]
    if len(fills) > len(free):
        for b in range(len(old)):
            at = int(old[b]) // page
            shared = new[b] > old[b] and old[b] % page and refs[table[b, at]] >= 2
            lacks = shared or held(new[b], page) > held(old[b], page)
            table[b, held(old[b], page):held(new[b], page)] = -1
            if lacks:
                new[b] = -1
        return False
    for (b, i), p in zip(fills, free):
        table[b, i] = p
        r[p] += 1
    for b, at, src in copies:
        for plane in planes:
            plane[table[b, at]] = plane[src]
    refs[:] = r
    return True


def free(refs, table, kv_len, page, rows):
    done = set()
    for b in (int(x) for x in rows):
        if b in done:
            continue
        done.add(b)
        for i in range(held(kv_len[b], page)):
            refs[table[b, i]] -= 1
        kv_len[b] = 0


def compact(refs, table, planes, page, kv_len):
    """Nothing moves where a length is out of range; entries whose page has no
    count stay."""
    if not all(0 <= n <= table.shape[1] * page for n in kv_len):
        return
    total = int((refs > 0).sum())
    src = [p for p in range(total, len(refs)) if refs[p] > 0]
    dst = [p for p in range(total) if refs[p] <= 0]
    for s, d in zip(src, dst):
        for plane in planes:
            plane[d] = plane[s]
        refs[d], refs[s] = refs[s], 0
    to = dict(zip(src, dst))
    for b in range(len(kv_len)):
        for i in range(held(kv_len[b], page)):
            table[b, i] = to.get(int(table[b, i]), table[b, i])
