"""Oracle of the paged cache's integer tables and of keeping an accepted path, in
plain Python: one sequence and one token at a time.  It shares no code with the
CUDA library.
"""

from __future__ import annotations

import numpy as np


def step(new_lens, lens, table, held, free, page, T, parents=None, words=1):
    """A step's tables.  `table` (rows of page numbers), `held` and `free` (the
    stack, last on top) are lists and change in place.  Returns a dict of cu_q,
    kv_lens, positions, slots, tree (None without parents)."""
    B = len(new_lens)
    for b in range(B):
        if new_lens[b] == -1:
            free.extend(table[b][:held[b]])
            held[b] = 0
    cu, kv = [0], []
    slots, positions = [-1] * T, [0] * T
    tree = np.zeros((T, words), np.uint32) if parents is not None else None
    short = full = False
    for b in range(B):
        n, m = max(0, new_lens[b]), lens[b]
        if short or cu[-1] + n > T:      # the call has no rows for it, nor for any later one
            short = True
            cu.append(cu[-1])
            kv.append(0 if new_lens[b] == -1 else m)
            continue
        need = 0 if new_lens[b] == -1 else max(0, -(-(m + n) // page) - held[b])
        room = need == 0 or (not full and need <= len(free))
        full = full or not room
        if room:
            for _ in range(need):
                table[b][held[b]] = free.pop()
                held[b] += 1
        kv.append(0 if new_lens[b] == -1 else m + n if room else m)
        for i in range(n):
            t = cu[-1] + i
            if room:
                slots[t] = table[b][(m + i) // page] * page + (m + i) % page
            positions[t] = m + i
            if parents is not None:
                seen = [i]
                while parents[cu[-1] + seen[-1]] >= 0:
                    seen.append(parents[cu[-1] + seen[-1]])
                positions[t] = m + len(seen) - 1
                for j in seen:
                    tree[t, j // 32] |= np.uint32(1 << (j % 32))
        cu.append(cu[-1] + n)
    return dict(cu_q=cu, kv_lens=kv, positions=positions, slots=slots,
                tree=None if tree is None else tree.view(np.int32))


def keep(cache, table, page, n, m, path):
    """Moves the nodes `path` of a sequence's n drafted tokens (the last of m) of
    one cache [pages, page, ...] behind its context, in place."""
    rows = [cache[table[(m - n + j) // page], (m - n + j) % page].copy() for j in path]
    for d, row in enumerate(rows):
        cache[table[(m - n + d) // page], (m - n + d) % page] = row
