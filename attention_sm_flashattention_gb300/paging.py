"""Python entry points of the paged cache's tables, kept on the GPU.

A pool of pages is a stack: ``free_pages`` int32 [num_pages] and its height
``free_count`` int32 [1] (``page_pool`` makes a full one).  ``cache_step`` takes
pages for the new tokens of a step and returns what ``rotary_and_cache`` (slots
and positions) and ``fwd_paged_scored`` (context lengths) need; ``cache_release``
gives the pages of finished sequences back.  Nothing is read back to the host,
so a loop's steps can be captured in a graph.  As in :mod:`.api`, these check
tensor metadata, allocate outputs and call the C ABI.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _native
from .api import _empty_on, _workspace
from .scored import _check_int, _elsewhere, _same_device, _stream


def page_pool(num_pages: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """``(free_pages, free_count)`` of a pool whose pages are all free; page 0
    is the first to go."""
    if num_pages < 1:
        raise ValueError("a pool has at least one page")
    return (torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
            torch.full((1,), num_pages, dtype=torch.int32, device=device))


_I32 = torch.int32


def _check_pool(free_pages, free_count, block_table, lens, name):
    """(B, num_pages, max_pages), checked; the quick look that most calls pass
    first (a call of the smallest sizes is bound by this module)."""
    if type(free_pages) is type(free_count) is type(block_table) is type(lens) is torch.Tensor:
        fs, cs, ts, ls = free_pages.shape, free_count.shape, block_table.shape, lens.shape
        if len(fs) == len(cs) == len(ls) == 1 and len(ts) == 2 and cs[0] == 1 and ls[0] == ts[0] > 0 and ts[1] > 0 \
                and fs[0] > 0 and free_pages.dtype is free_count.dtype is block_table.dtype is lens.dtype is _I32 \
                and free_pages.is_cuda and free_count.is_cuda and block_table.is_cuda and lens.is_cuda \
                and free_pages.is_contiguous() and block_table.is_contiguous() and lens.is_contiguous():
            return ts[0], fs[0], ts[1]
    for n, t, dims in (("free_pages", free_pages, 1), ("block_table", block_table, 2), (name, lens, 1)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{n} must be an int32 CUDA tensor of {dims} dimension{'s' * (dims > 1)}")
    B, max_pages = block_table.shape
    _check_int("free_pages", free_pages, torch.int32, free_pages.shape)
    _check_int("free_count", free_count, torch.int32, (1,))
    _check_int("block_table", block_table, torch.int32, (B, max_pages))
    _check_int(name, lens, torch.int32, (B,))
    if B < 1 or max_pages < 1 or free_pages.shape[0] < 1:
        raise ValueError("the tables need at least one sequence, page per sequence and page in the pool")
    return B, free_pages.shape[0], max_pages


def _apart(out, taken) -> None:
    """Outputs may not overlap each other, or any of the inputs of ``taken`` but
    the one (same address) that they may replace."""
    spans = []
    for name, t, may_be in out:
        at, end = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        for other, o in taken:
            if o is None or (other == may_be and o.data_ptr() == at):
                continue
            if at < o.data_ptr() + o.numel() * o.element_size() and o.data_ptr() < end:
                raise ValueError(f"out: {name} overlaps {other}")
        if any(at < b and a < end for a, b in spans):
            raise ValueError(f"out: {name} overlaps another output")
        spans.append((at, end))


def cache_step(free_pages: torch.Tensor, free_count: torch.Tensor, block_table: torch.Tensor,
               cached_lens: torch.Tensor, q_lens: Optional[torch.Tensor], N: int, page_size: int,
               out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]] = None,
               stream: Optional[torch.cuda.Stream] = None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Pages, slots and positions of a step's new tokens.  ``cached_lens`` int32
    [B]: tokens that each sequence has; ``q_lens`` int32 [B]: its new ones, at
    most N (None: N); ``block_table`` int32 [B, max_pages]: the entries of the
    pages that begin with new tokens are written, taken from the top of the
    stack in the order of sequences and pages.  Returns ``(slot_mapping,
    positions, context_lens, free_count)``: int64 [B, N] slots (-1 behind the
    new tokens, past max_pages and where a page is missing), int64 [B, N]
    positions, int32 [B] lengths with the new tokens, int32 [1] the stack's
    height (negative: so many pages were missing).  ``out``: the four, where the
    last two may be ``cached_lens`` and ``free_count`` themselves.

    The new lengths count tokens without a slot too.  A sequence that outgrows
    its max_pages pages has to end before: attention clamps lengths to the table
    and would take its last rows for earlier positions."""
    B, num_pages, max_pages = _check_pool(free_pages, free_count, block_table, cached_lens, "cached_lens")
    if N < 1 or page_size < 1 or N > 0x7fffffff or page_size > 0x7fffffff:
        raise ValueError(f"N and page_size must be positive 32-bit numbers, got {N} and {page_size}")
    if q_lens is not None:
        _check_int("q_lens", q_lens, torch.int32, (B,))
    if _elsewhere(free_pages):
        with torch.cuda.device(free_pages.device):
            return cache_step(free_pages, free_count, block_table, cached_lens, q_lens, N, page_size, out, stream)
    handle = _stream(_same_device(free_pages, free_count, block_table, cached_lens, q_lens), stream)
    if out is None and stream is None:
        slots = torch.empty((B, N), dtype=torch.int64, device=free_pages.device)
        out = slots, torch.empty_like(slots), torch.empty_like(cached_lens), torch.empty_like(free_count)
    elif out is None:
        out = _empty_on(stream, free_pages.device, ((B, N), torch.int64), ((B, N), torch.int64), ((B,), torch.int32),
                        ((1,), torch.int32))
    else:
        for name, t, dtype, shape in zip(("slot_mapping", "positions", "context_lens", "free_count"), out,
                                         (torch.int64, torch.int64, torch.int32, torch.int32),
                                         ((B, N), (B, N), (B,), (1,))):
            _check_int("out: " + name, t, dtype, shape)
        _same_device(free_pages, *out)
        _apart((("slot_mapping", out[0], None), ("positions", out[1], None), ("context_lens", out[2], "cached_lens"),
                ("free_count", out[3], "free_count"), ("block_table", block_table, "block_table")),
               (("free_pages", free_pages), ("free_count", free_count), ("block_table", block_table),
                ("cached_lens", cached_lens), ("q_lens", q_lens)))
    slots, positions, context_lens, count = out
    rc = _native.lib().fa_cache_step(free_pages.data_ptr(), free_count.data_ptr(), block_table.data_ptr(),
                                     cached_lens.data_ptr(), q_lens.data_ptr() if q_lens is not None else None,
                                     slots.data_ptr(), positions.data_ptr(), context_lens.data_ptr(), count.data_ptr(),
                                     B, N, num_pages, page_size, max_pages, handle)
    _native.check(rc, "fa_cache_step")
    return slots, positions, context_lens, count


def cache_release(free_pages: torch.Tensor, free_count: torch.Tensor, block_table: torch.Tensor,
                  context_lens: torch.Tensor, finished: torch.Tensor, page_size: int,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                  stream: Optional[torch.cuda.Stream] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gives back the pages of the sequences where ``finished`` (bool [B]) is
    set: the valid entries of their first ``context_lens`` tokens go onto the
    stack in the order of sequences and pages.  Returns ``(context_lens,
    free_count)``: 0 for those sequences, and the stack's new height; ``out``:
    the two, which may be the inputs themselves.  The block table is left as it
    is.  ``workspace``: 4 (B + 1) bytes.

    Pages are given back by whole sequences alone: those that a window has
    passed stay with a running sequence until it ends.  A page belongs to one
    sequence: one that the rows of two name (a shared prefix) goes onto the
    stack twice, and would be handed out twice."""
    B, num_pages, max_pages = _check_pool(free_pages, free_count, block_table, context_lens, "context_lens")
    _check_int("finished", finished, torch.bool, (B,))
    if page_size < 1 or page_size > 0x7fffffff:
        raise ValueError(f"page_size must be a positive 32-bit number, got {page_size}")
    if _elsewhere(free_pages):
        with torch.cuda.device(free_pages.device):
            return cache_release(free_pages, free_count, block_table, context_lens, finished, page_size, out, stream,
                                 workspace)
    handle = _stream(_same_device(free_pages, free_count, block_table, context_lens, finished, workspace), stream)
    lib = _native.lib()
    if workspace is None:
        workspace, = _empty_on(stream, free_pages.device, (B + 1, torch.int32), result=False)
    if out is None and stream is None:
        out = torch.empty_like(context_lens), torch.empty_like(free_count)
    elif out is None:
        out = _empty_on(stream, free_pages.device, ((B,), torch.int32), ((1,), torch.int32))
    else:
        _check_int("out: context_lens", out[0], torch.int32, (B,))
        _check_int("out: free_count", out[1], torch.int32, (1,))
        _same_device(free_pages, *out)
        _apart((("context_lens", out[0], "context_lens"), ("free_count", out[1], "free_count"),
                ("free_pages", free_pages, "free_pages"), ("workspace", workspace, None)),
               (("free_pages", free_pages), ("free_count", free_count), ("block_table", block_table),
                ("context_lens", context_lens), ("finished", finished)))
    lens, count = out
    rc = lib.fa_cache_release(free_pages.data_ptr(), free_count.data_ptr(), block_table.data_ptr(),
                              context_lens.data_ptr(), finished.data_ptr(), lens.data_ptr(), count.data_ptr(),
                              *_workspace(workspace), B, num_pages, page_size, max_pages, handle)
    _native.check(rc, "fa_cache_release")
    return lens, count
