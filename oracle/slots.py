"""Block tables and slot maps from request lengths, one sequence at a time.

A sequence of P + n tokens wants ceil((P + n) / 16) blocks; what it does not
hold is popped from the free list (a stack), in sequence order and then table
order.  The sequences are served in order as long as the needs so far fit;
from the first one that does not fit on, only sequences that need nothing are
served.  Releasing pushes blocks so that it undoes the pops exactly (a popped id
that names no block of the pool is -1 in the table, and comes back as that).
"""

from __future__ import annotations

import numpy as np

PAGE = 16
BAD_PAGE, BAD_LEN, NO_BLOCK = 1, 2, 16


def slots_build(prefix_len, n_new, N_max, block_table, held, free_list, free_count):
    """Returns (slots, block_table, held, free_count, status), inputs unchanged."""
    table, held = np.array(block_table), np.array(held)
    B, max_blocks = table.shape
    num_blocks = len(free_list)
    count = int(free_count)
    slots = np.full((B, N_max), -1, dtype=np.int32)
    status = 0
    count_ok = 0 <= count <= num_blocks
    if not count_ok:
        status |= BAD_LEN
    total = 0
    top = count
    for b in range(B):
        P, n = int(prefix_len[b]), int(n_new[b]) if n_new is not None else N_max
        if P < 0 or n < 0 or n > N_max or P + n > max_blocks * PAGE or not 0 <= held[b] <= max_blocks:
            status |= BAD_LEN
            continue
        want = -(-(P + n) // PAGE)
        need = max(0, want - int(held[b]))
        total += need
        if need and (not count_ok or total > count):
            if count_ok:
                status |= NO_BLOCK
            continue
        for j in range(int(held[b]), want):
            top -= 1
            page = int(free_list[top])
            if not 0 <= page < num_blocks:
                status |= BAD_PAGE
                page = -1
            table[b, j] = page
        held[b] = max(int(held[b]), want)
        for i in range(n):
            page = int(table[b, (P + i) // PAGE])
            if not 0 <= page < num_blocks:
                status |= BAD_PAGE
                continue
            slots[b, i] = page * PAGE + (P + i) % PAGE
    return slots, table, held, top if count_ok else count, status


def blocks_release(keep_len, block_table, held, free_list, free_count):
    """Returns (block_table, held, free_list, free_count, status)."""
    table, held, free = np.array(block_table), np.array(held), np.array(free_list)
    B, max_blocks = table.shape
    count, status = int(free_count), 0
    given = []
    after = held.copy()
    for b in range(B):
        if keep_len[b] < 0 or not 0 <= held[b] <= max_blocks:
            status |= BAD_LEN
            continue
        want = -(-int(keep_len[b]) // PAGE)
        for j in range(want, int(held[b])):
            given.append((b, j))
        after[b] = min(int(held[b]), want)
    if not 0 <= count <= len(free) or len(given) > len(free) - count:
        return table, held, free, count, status | BAD_LEN
    for i, (b, j) in enumerate(given):
        if not 0 <= table[b, j] < len(free):
            status |= BAD_PAGE
        free[count + len(given) - 1 - i] = table[b, j]
        table[b, j] = -1
    return table, after, free, count + len(given), status
