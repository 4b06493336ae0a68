"""Page sharing, freeing and compaction on a block table, one row and one page at a time.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

The table is the only state: page p is in use while some row has it among its first
ceil(length / page_size) entries.  Readings: see ``include/attn_b200.h`` (attn_pages_fork,
attn_pages_compact); this module follows them in the plainest sequential way.
"""

from __future__ import annotations

import numpy as np


def fork(table, lens, parents, add, new_cols: int, page_size: int, num_pages: int):
    """(new table, new lengths, free pages left, copies as (source, destination), pages ran out)."""
    rows, kept_lens, new_lens = [], [], []
    for i, p in enumerate(parents):
        if p < 0:
            rows.append([])
            kept_lens.append(0)
            new_lens.append(0)
            continue
        old = int(lens[p])
        new = old + (0 if add is None else int(add[i]))
        if new < 0 or new > new_cols * page_size:
            new = old
        kept = min(old, new)
        rows.append([int(e) for e in table[p][: -(-kept // page_size)]])
        kept_lens.append(kept)
        new_lens.append(new)
    in_use = {e for r in rows for e in r}
    full = {e for r, n in zip(rows, kept_lens) for e in r[: n // page_size]}
    free = [p for p in range(num_pages) if p not in in_use]
    taken, owned, copies, short = 0, set(), [], False
    for r, kept, new in zip(rows, kept_lens, new_lens):
        def fresh():
            nonlocal taken, short
            taken += 1
            if taken > len(free):
                short = True
                return -1
            return free[taken - 1]

        if kept % page_size:
            e = r[-1]
            if e in full or e in owned:
                r[-1] = fresh()
                if r[-1] >= 0:
                    copies.append((e, r[-1]))
            owned.add(e)
        while len(r) < -(-new // page_size):
            r.append(fresh())
    out = np.full((len(parents), new_cols), -1, dtype=np.int32)
    for i, r in enumerate(rows):
        out[i, : len(r)] = r
    return out, np.array(new_lens, dtype=np.int32), max(0, len(free) - taken), copies, short


def compact(table, lens, page_size: int, num_pages: int):
    """(new table, page map, pages in use, moves as (source, destination))."""
    used = [-(-int(n) // page_size) for n in lens]
    live = sorted({int(e) for r, n in zip(table, used) for e in r[:n]})
    holes = [p for p in range(len(live)) if p not in set(live)]
    movers = [p for p in live if p >= len(live)]
    page_map = np.full(num_pages, -1, dtype=np.int32)
    for p in live:
        page_map[p] = p
    for src, dst in zip(movers, holes):
        page_map[src] = dst
    out = np.full(np.shape(table), -1, dtype=np.int32)
    for i, n in enumerate(used):
        out[i, :n] = page_map[np.asarray(table[i][:n], dtype=np.int64)]
    return out, page_map, len(live), list(zip(movers, holes))
