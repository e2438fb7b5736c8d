"""The page tables' rules, token by token in plain Python."""

from __future__ import annotations


def _clamp(x, lo, hi):
    return min(max(int(x), lo), hi)


def step(free_pages, free_count, block_table, cached_lens, q_lens, N, page_size):
    """(slots, positions, context_lens, free_count, block_table) as lists, after a step; the inputs are left alone."""
    pages, table = len(free_pages), [[int(x) for x in row] for row in block_table]
    height = top = _clamp(free_count, 0, pages)
    slots, positions, lens = [], [], []
    for b, row in enumerate(table):
        have = max(int(cached_lens[b]), 0)
        new = N if q_lens is None else _clamp(q_lens[b], 0, N)
        slots.append([])
        positions.append([have + n for n in range(N)])
        for n in range(N):
            p = have + n
            at = p // page_size
            if n >= new or at >= len(row):
                slots[-1].append(-1)
                continue
            if p % page_size == 0:  # a new page
                top -= 1
                row[at] = int(free_pages[top]) if top >= 0 else -1
            slots[-1].append(row[at] * page_size + p % page_size if 0 <= row[at] < pages else -1)
        lens.append(min(have + new, 2 ** 31 - 1))
    assert top <= height
    return slots, positions, lens, top, table


def release(free_pages, free_count, block_table, context_lens, finished, page_size):
    """(context_lens, free_count, free_pages) as lists, after giving back."""
    pages, stack = len(free_pages), [int(x) for x in free_pages]
    top, lens = _clamp(free_count, 0, pages), []
    for b, row in enumerate(block_table):
        held = -(-max(int(context_lens[b]), 0) // page_size)
        for x in row[:held] if finished[b] else ():
            if 0 <= int(x) < pages and top < pages:
                stack[top] = int(x)
                top += 1
        lens.append(0 if finished[b] else int(context_lens[b]))
    return lens, top, stack
