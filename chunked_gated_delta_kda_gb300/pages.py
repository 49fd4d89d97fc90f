"""Pages that several requests own (argument marshalling only).

Beside ``latent.block_tables``, which takes pages from the free list:

``page_fork``     requests that go on from another one's tokens share its pages,
``page_copy``     copies pages in the caches of all layers (or in pools of states),
``page_free``     gives back the pages behind the tokens that a request keeps,
``page_compact``  brings the pages in use onto the lowest numbers.

``refs`` (int32, a number for each page) is how many owners a page has beside
its first, so pages that ``block_tables`` takes need no entry.  Every step runs
in the kernels of ``libkda.so`` (``include/kda.h`` has the contract); this
module checks torch tensors, allocates outputs on the tensors' device and
passes pointers and torch's current stream.  If the library is missing, every
call raises: there is no fallback path.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from .binding import load_library
from .latent import (INT_MAX, _check, _check_int, _current_device, _elsewhere, _hand_back, _raise, _same_device, _scratch,
                     _status_workspace, _stream, _together)


def _checked(block_table, seq_lens, refs, free_pages, free_head, page_size, rows=(), vectors=()):
    """Checks what the three table functions share; ``rows``: more (name, tensor) pairs of seq_lens' shape, ``vectors``:
    of any length."""
    try:
        fine = (block_table.dtype is seq_lens.dtype is refs.dtype is free_pages.dtype is free_head.dtype is torch.int32
                and block_table.dim() == 2 and refs.dim() == free_pages.dim() == 1 and free_head.shape == (1,)
                and seq_lens.shape == block_table.shape[:1] and 0 < page_size <= INT_MAX and page_size % 1 == 0
                and all(t.dtype is torch.int32 and t.shape == seq_lens.shape for _, t in rows)
                and all(t.dtype is torch.int32 and t.dim() == 1 for _, t in vectors)
                and max(block_table.size(0), block_table.size(1), refs.size(0), free_pages.size(0)) <= INT_MAX
                and _together(seq_lens.get_device(), block_table, refs, free_pages, free_head, *(t for _, t in rows),
                              *(t for _, t in vectors)))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check_int("page_size", page_size)
        if page_size < 1:
            raise ValueError(f"page_size must be positive, got {page_size}")
        _check("block_table", block_table, torch.int32, (None, None))
        _check("seq_lens", seq_lens, torch.int32, (block_table.shape[0],))
        _check("refs", refs, torch.int32, (None,))
        _check("free_pages", free_pages, torch.int32, (None,))
        _check("free_head", free_head, torch.int32, (1,))
        for name, t in rows:
            _check(name, t, torch.int32, seq_lens.shape)
        for name, t in vectors:
            _check(name, t, torch.int32, (None,))
        for name, t in (("block_table", block_table), ("refs", refs), ("free_pages", free_pages)):
            for size in t.shape:
                _check_int(f"a size of {name}", size)
        _same_device(seq_lens.get_device(), block_table, refs, free_pages, free_head, *(t for _, t in rows),
                     *(t for _, t in vectors))


def page_fork(block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
              refs: torch.Tensor, free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int,
              workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Rows ``children[i]`` of the table go on from the tokens of rows ``parents[i]``.

    block_table: int32 [N, width], the children's cells are written in place;
    seq_lens: int32 [N]; parents, children: int32 [F] (a negative child is
    skipped), the children distinct rows of length 0; refs: int32 [pages];
    free_pages: int32 [free] and free_head: int32 [1], as for ``block_tables``.
    Full pages are shared; a last page that is not full gets a page of its own.
    Returns (the new lengths, the new refs, the new free_head, pairs int32
    [F, 2] for ``page_copy``: the page to copy and the own page, or -1); the
    other inputs stay as they are.  ``workspace`` (256-byte aligned,
    ``page_fork_workspace_bytes``) records device-detected faults for
    ``binding.get_status``; beside a smaller one another is allocated."""
    _checked(block_table, seq_lens, refs, free_pages, free_head, page_size, vectors=(("parents", parents), ("children", children)))
    if parents.shape != children.shape or parents.shape[0] > INT_MAX:
        raise ValueError(f"parents and children must be of one length, got {parents.shape[0]} and {children.shape[0]}")
    index = seq_lens.get_device()
    if index != _current_device():
        return _elsewhere(index, page_fork, block_table, seq_lens, parents, children, refs, free_pages, free_head, page_size,
                          workspace)
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    # copies are held until the launch: a freed one's memory would go to the next
    seq_lens, refs, free_pages = seq_lens.contiguous(), refs.contiguous(), free_pages.contiguous()
    parents, children = parents.contiguous(), children.contiguous()
    (N, width), F = block_table.shape, parents.shape[0]
    scratch = _scratch(workspace, page_fork_workspace_bytes(N), index, seq_lens.device)
    lens_out, refs_out, head_out = torch.empty_like(seq_lens), torch.empty_like(refs), torch.empty_like(free_head)
    pairs = torch.empty((F, 2), dtype=torch.int32, device=seq_lens.device)
    _raise(load_library().kda_page_fork(
        block_table.data_ptr(), width, seq_lens.data_ptr(), parents.data_ptr(), children.data_ptr(), refs.data_ptr(),
        refs.shape[0], free_pages.data_ptr(), free_pages.shape[0], free_head.data_ptr(), int(page_size), lens_out.data_ptr(),
        refs_out.data_ptr(), head_out.data_ptr(), pairs.data_ptr(), N, F, scratch.data_ptr(),
        scratch.numel() * scratch.element_size(), _stream(index)), "kda_page_fork")
    _hand_back(scratch, workspace)
    return lens_out, refs_out, head_out, pairs


def page_fork_workspace_bytes(N: int) -> int:
    return int(load_library().kda_page_fork_workspace_bytes(N))


def page_free_workspace_bytes(pages: int) -> int:
    return int(load_library().kda_page_free_workspace_bytes(pages))


def page_compact_workspace_bytes(pages: int) -> int:
    return int(load_library().kda_page_compact_workspace_bytes(pages))


def page_copy(pools: Union[torch.Tensor, Sequence[torch.Tensor]], pairs: torch.Tensor,
              count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Copy pages within each pool: page ``pairs[i, 1]`` becomes page ``pairs[i, 0]``.

    pools: a tensor [pages, ...] or several of one shape and type (the caches
    of all layers, or pools of states), contiguous, pages of a multiple of 16
    bytes; pairs: int32 [F, 2], a pair with a negative entry is skipped; the
    targets distinct, and none of them a source; count: int32 [1] on the
    device, how many pairs count (None: all).  ``workspace`` (256 bytes,
    256-byte aligned) records device-detected faults.  Returns ``pools``,
    updated in place."""
    if not isinstance(pools, (torch.Tensor, list, tuple)):
        raise TypeError("pools must be a torch.Tensor or a list of them")
    several = [pools] if isinstance(pools, torch.Tensor) else pools
    if not several:
        raise ValueError("pools must not be empty")
    first = several[0]
    for t in several:
        if not isinstance(t, torch.Tensor):
            raise TypeError("pools must be torch.Tensors")
        if not t.is_cuda or t.dim() < 1 or not t.is_contiguous():
            raise ValueError(f"pools must be contiguous CUDA tensors [pages, ...], got {tuple(t.shape)} on {t.device}")
        if t.shape != first.shape or t.dtype is not first.dtype:
            raise ValueError("pools must have one shape and type")
    _check("pairs", pairs, torch.int32, (None, 2))
    if count is not None:
        _check("count", count, torch.int32, (1,))
    _check_int("a size of pairs", pairs.shape[0])
    _check_int("a size of pools", first.shape[0])
    index = first.get_device()
    _same_device(index, pairs, count, *several)
    if index != _current_device():
        return _elsewhere(index, page_copy, pools, pairs, count, workspace)
    pages = first.shape[0]
    page_bytes = first.numel() // max(pages, 1) * first.element_size()
    if pages < 1 or page_bytes < 16 or page_bytes % 16 or any(t.data_ptr() % 16 for t in several):
        raise ValueError(f"pools need pages of a multiple of 16 bytes that start on 16 bytes, got {pages} of {page_bytes}")
    pairs = pairs.contiguous()
    at = (ctypes.c_void_p * len(several))(*[t.data_ptr() for t in several])
    _raise(load_library().kda_page_copy(at, len(several), pages, page_bytes, pairs.data_ptr(),
                                        None if count is None else count.data_ptr(), pairs.shape[0],
                                        _status_workspace(workspace, index), _stream(index)), "kda_page_copy")
    return pools


def page_free(block_table: torch.Tensor, seq_lens: torch.Tensor, keep_lens: torch.Tensor, refs: torch.Tensor,
              free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int, workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Row n of the table keeps its first ``keep_lens[n]`` tokens (0: the request ends; fewer than it has: rejected drafts).

    block_table: int32 [N, width]; seq_lens, keep_lens: int32 [N], keep_lens at
    most seq_lens; refs: int32 [pages]; free_pages: int32 [free] and free_head:
    int32 [1].  The pages that lose their last owner come in front of the free
    list, in increasing order: their entries of ``free_pages`` are written in
    place.  Returns (the new lengths, the new refs, the new free_head); the
    other inputs stay as they are.  ``workspace`` as for ``page_fork``, with
    ``page_free_workspace_bytes`` bytes."""
    _checked(block_table, seq_lens, refs, free_pages, free_head, page_size, rows=(("keep_lens", keep_lens),))
    index = seq_lens.get_device()
    if index != _current_device():
        return _elsewhere(index, page_free, block_table, seq_lens, keep_lens, refs, free_pages, free_head, page_size, workspace)
    if not free_pages.is_contiguous():
        raise ValueError("free_pages must be contiguous")
    block_table, seq_lens, keep_lens, refs = (t.contiguous() for t in (block_table, seq_lens, keep_lens, refs))
    (N, width), pages = block_table.shape, refs.shape[0]
    scratch = _scratch(workspace, page_free_workspace_bytes(pages), index, seq_lens.device)
    lens_out, refs_out, head_out = torch.empty_like(seq_lens), torch.empty_like(refs), torch.empty_like(free_head)
    _raise(load_library().kda_page_free(
        block_table.data_ptr(), width, seq_lens.data_ptr(), keep_lens.data_ptr(), refs.data_ptr(), pages,
        free_pages.data_ptr(), free_pages.shape[0], free_head.data_ptr(), int(page_size), lens_out.data_ptr(),
        refs_out.data_ptr(), head_out.data_ptr(), N, scratch.data_ptr(), scratch.numel() * scratch.element_size(),
        _stream(index)), "kda_page_free")
    _hand_back(scratch, workspace)
    return lens_out, refs_out, head_out


def page_compact(block_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor, free_pages: torch.Tensor,
                 free_head: torch.Tensor, page_size: int, workspace: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """The U pages that are not in the free list onto the numbers 0 .. U - 1: those from U on move, in increasing order,
    to the free pages below U.

    Arguments as for ``page_free``.  Returns (the new block_table, -1 behind a
    row's pages; the new refs; the new free_pages, U, U + 1, ... from free_head
    on, which stays; pairs int32 [pages // 2, 2] and count int32 [1] for
    ``page_copy``; moved int32 [pages], each page's new number, -1 for a free
    one).  The inputs stay as they are: copy the pages of every cache before
    the new table is used.  ``workspace`` as for ``page_fork``, with
    ``page_compact_workspace_bytes`` bytes."""
    _checked(block_table, seq_lens, refs, free_pages, free_head, page_size)
    index = seq_lens.get_device()
    if index != _current_device():
        return _elsewhere(index, page_compact, block_table, seq_lens, refs, free_pages, free_head, page_size, workspace)
    block_table, seq_lens, refs, free_pages = (t.contiguous() for t in (block_table, seq_lens, refs, free_pages))
    (N, width), pages = block_table.shape, refs.shape[0]
    scratch = _scratch(workspace, page_compact_workspace_bytes(pages), index, seq_lens.device)
    table_out, refs_out, free_out = torch.empty_like(block_table), torch.empty_like(refs), torch.empty_like(free_pages)
    pairs = torch.empty((pages // 2, 2), dtype=torch.int32, device=seq_lens.device)
    count, moved = torch.empty_like(free_head), torch.empty_like(refs)
    _raise(load_library().kda_page_compact(
        block_table.data_ptr(), width, seq_lens.data_ptr(), refs.data_ptr(), pages, free_pages.data_ptr(),
        free_pages.shape[0], free_head.data_ptr(), int(page_size), table_out.data_ptr(), refs_out.data_ptr(),
        free_out.data_ptr(), pairs.data_ptr(), count.data_ptr(), moved.data_ptr(), N, scratch.data_ptr(),
        scratch.numel() * scratch.element_size(), _stream(index)), "kda_page_compact")
    _hand_back(scratch, workspace)
    return table_out, refs_out, free_out, pairs, count, moved
