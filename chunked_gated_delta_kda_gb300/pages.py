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
from .latent import INT_MAX, _check, _check_int, _current_device, _elsewhere, _raise, _same_device, _status_workspace, _stream, _together

_I32 = torch.int32


def _explain(block_table, seq_lens, refs, free_pages, free_head, page_size, **more):
    """Says what is wrong with the arguments of a table function (see ``latent``'s checks); ``more``: tensors of
    seq_lens' length, or with a name that ends in ``s_`` of any."""
    _check_int("page_size", page_size)
    if page_size < 1:
        raise ValueError(f"page_size must be positive, got {page_size}")
    _check("block_table", block_table, _I32, (None, None))
    _check("seq_lens", seq_lens, _I32, (block_table.shape[0],))
    _check("refs", refs, _I32, (None,))
    _check("free_pages", free_pages, _I32, (None,))
    _check("free_head", free_head, _I32, (1,))
    for name, t in more.items():
        _check(name.rstrip("_"), t, _I32, (None,) if name[-1] == "_" else (block_table.shape[0],))
    for name, t in (("block_table", block_table), ("refs", refs), ("free_pages", free_pages), *more.items()):
        for size in t.shape:
            _check_int(f"a size of {name.rstrip('_')}", size)
    _same_device(seq_lens.get_device(), block_table, refs, free_pages, free_head, *more.values())


def page_fork(block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
              refs: torch.Tensor, free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int,
              fork_lens: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Rows ``children[i]`` of the table go on from the tokens of rows ``parents[i]``.

    block_table: int32 [N, width], the children's cells are written in place;
    seq_lens: int32 [N]; parents, children: int32 [F] (a negative child is
    skipped), the children distinct rows of length 0; refs: int32 [pages];
    free_pages: int32 [free] and free_head: int32 [1], as for ``block_tables``;
    fork_lens: int32 [F], how many of the parent's first tokens (None: all).
    Full pages are shared; a last page that is not full gets a page of its own.
    Returns (the new lengths, the new refs, the new free_head, pairs int32
    [F, 2] for ``page_copy``: the page to copy and the own page, or -1); the
    other inputs stay as they are.  ``workspace`` (256 bytes, 256-byte aligned)
    records device-detected faults for ``binding.get_status``."""
    try:
        index = seq_lens.get_device()
        N, width = block_table.shape
        (pages,), (free,), (F,) = refs.shape, free_pages.shape, parents.shape
        fine = (block_table.dtype is seq_lens.dtype is parents.dtype is children.dtype is refs.dtype is free_pages.dtype
                is free_head.dtype is _I32 and seq_lens.shape == (N,) and children.shape == (F,) and free_head.shape == (1,)
                and (fork_lens is None or fork_lens.dtype is _I32 and fork_lens.shape == (F,))
                and 0 < page_size <= INT_MAX and page_size % 1 == 0 and max(N, width, pages, free, F) <= INT_MAX
                and _together(index, block_table, parents, children, fork_lens, refs, free_pages, free_head))
    except (AttributeError, ValueError):   # not a tensor, or not of one dimension or two
        fine = False
    if not fine:
        more = {} if fork_lens is None else dict(fork_lens_=fork_lens)
        _explain(block_table, seq_lens, refs, free_pages, free_head, page_size, parents_=parents, children_=children, **more)
        raise ValueError("parents, children and fork_lens must be of one length, got "
                         f"{[t.shape[0] for t in (parents, children, *more.values())]}")
    if index != _current_device():
        return _elsewhere(index, page_fork, block_table, seq_lens, parents, children, refs, free_pages, free_head, page_size,
                          fork_lens, workspace)
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    # copies are held until the launch: a freed one's memory would go to the next
    seq_lens, refs, free_pages = seq_lens.contiguous(), refs.contiguous(), free_pages.contiguous()
    parents, children = parents.contiguous(), children.contiguous()
    if fork_lens is not None:
        fork_lens = fork_lens.contiguous()
    lens_out, refs_out, head_out = torch.empty_like(seq_lens), torch.empty_like(refs), torch.empty_like(free_head)
    pairs = torch.empty((F, 2), dtype=_I32, device=seq_lens.device)
    _raise(load_library().kda_page_fork(
        block_table.data_ptr(), width, seq_lens.data_ptr(), parents.data_ptr(), children.data_ptr(),
        None if fork_lens is None else fork_lens.data_ptr(), refs.data_ptr(), pages,
        free_pages.data_ptr(), free, free_head.data_ptr(), int(page_size), lens_out.data_ptr(), refs_out.data_ptr(),
        head_out.data_ptr(), pairs.data_ptr(), N, F, _status_workspace(workspace, index), _stream(index)), "kda_page_fork")
    return lens_out, refs_out, head_out, pairs


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
    several = (pools,) if isinstance(pools, torch.Tensor) else pools
    if not several:
        raise ValueError("pools must not be empty")
    first = several[0]
    try:
        index, shape, dtype = first.get_device(), first.shape, first.dtype
        fine = (pairs.dtype is _I32 and pairs.dim() == 2 and pairs.shape[1] == 2 and len(shape) > 0
                and (count is None or count.dtype is _I32 and count.shape == (1,))
                and max(pairs.shape[0], shape[0]) <= INT_MAX and _together(index, pairs, count))
        at, low = [], 0
        for t in several:
            fine = fine and t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            at.append(t.data_ptr())
            low |= at[-1]
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        for t in several:
            if not isinstance(t, torch.Tensor):
                raise TypeError("pools must be torch.Tensors")
            if not t.is_cuda or t.dim() < 1 or not t.is_contiguous():
                raise ValueError(f"pools must be contiguous CUDA tensors [pages, ...], got {tuple(t.shape)} on {t.device}")
            if t.shape != first.shape or t.dtype is not first.dtype:
                raise ValueError("pools must have one shape and type")
        _check("pairs", pairs, _I32, (None, 2))
        if count is not None:
            _check("count", count, _I32, (1,))
        _check_int("a size of pairs", pairs.shape[0])
        _check_int("a size of pools", first.shape[0])
        _same_device(first.get_device(), pairs, count, *several)
    if index != _current_device():
        return _elsewhere(index, page_copy, pools, pairs, count, workspace)
    pages = shape[0]
    page_bytes = first.numel() // max(pages, 1) * first.element_size()
    if pages < 1 or page_bytes < 16 or page_bytes % 16 or low % 16:
        raise ValueError(f"pools must have pages of a multiple of 16 bytes that start on 16 bytes, got {pages} of {page_bytes}")
    pairs = pairs.contiguous()
    _raise(load_library().kda_page_copy((ctypes.c_void_p * len(at))(*at), len(at), pages, page_bytes, pairs.data_ptr(),
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
    other inputs stay as they are.  A row that goes back into a page that has
    another owner left is reported: tokens appended to it would overwrite that
    one's (``page_fork`` its first tokens into another row instead).
    ``workspace`` as for ``page_fork``."""
    try:
        index = seq_lens.get_device()
        N, width = block_table.shape
        (pages,), (free,) = refs.shape, free_pages.shape
        fine = (block_table.dtype is seq_lens.dtype is keep_lens.dtype is refs.dtype is free_pages.dtype is free_head.dtype is _I32
                and seq_lens.shape == keep_lens.shape == (N,) and free_head.shape == (1,)
                and 0 < page_size <= INT_MAX and page_size % 1 == 0 and max(N, width, pages, free) <= INT_MAX
                and _together(index, block_table, keep_lens, refs, free_pages, free_head))
    except (AttributeError, ValueError):   # not a tensor, or not of one dimension or two
        fine = False
    if not fine:
        _explain(block_table, seq_lens, refs, free_pages, free_head, page_size, keep_lens=keep_lens)
    if index != _current_device():
        return _elsewhere(index, page_free, block_table, seq_lens, keep_lens, refs, free_pages, free_head, page_size, workspace)
    if not free_pages.is_contiguous():
        raise ValueError("free_pages must be contiguous")
    block_table, seq_lens, keep_lens, refs = block_table.contiguous(), seq_lens.contiguous(), keep_lens.contiguous(), refs.contiguous()
    lens_out, refs_out, head_out = torch.empty_like(seq_lens), torch.empty_like(refs), torch.empty_like(free_head)
    _raise(load_library().kda_page_free(
        block_table.data_ptr(), width, seq_lens.data_ptr(), keep_lens.data_ptr(), refs.data_ptr(), pages, free_pages.data_ptr(),
        free, free_head.data_ptr(), int(page_size), lens_out.data_ptr(), refs_out.data_ptr(), head_out.data_ptr(), N,
        _status_workspace(workspace, index), _stream(index)), "kda_page_free")
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
    the new table is used.  ``workspace`` as for ``page_fork``."""
    try:
        index = seq_lens.get_device()
        N, width = block_table.shape
        (pages,), (free,) = refs.shape, free_pages.shape
        fine = (block_table.dtype is seq_lens.dtype is refs.dtype is free_pages.dtype is free_head.dtype is _I32
                and seq_lens.shape == (N,) and free_head.shape == (1,)
                and 0 < page_size <= INT_MAX and page_size % 1 == 0 and max(N, width, pages, free) <= INT_MAX
                and _together(index, block_table, refs, free_pages, free_head))
    except (AttributeError, ValueError):   # not a tensor, or not of one dimension or two
        fine = False
    if not fine:
        _explain(block_table, seq_lens, refs, free_pages, free_head, page_size)
    if index != _current_device():
        return _elsewhere(index, page_compact, block_table, seq_lens, refs, free_pages, free_head, page_size, workspace)
    block_table, seq_lens, refs, free_pages = block_table.contiguous(), seq_lens.contiguous(), refs.contiguous(), free_pages.contiguous()
    table_out, refs_out, free_out = torch.empty_like(block_table), torch.empty_like(refs), torch.empty_like(free_pages)
    pairs = torch.empty((pages // 2, 2), dtype=_I32, device=seq_lens.device)
    count, moved = torch.empty_like(free_head), torch.empty_like(refs)
    _raise(load_library().kda_page_compact(
        block_table.data_ptr(), width, seq_lens.data_ptr(), refs.data_ptr(), pages, free_pages.data_ptr(), free,
        free_head.data_ptr(), int(page_size), table_out.data_ptr(), refs_out.data_ptr(), free_out.data_ptr(), pairs.data_ptr(),
        count.data_ptr(), moved.data_ptr(), N, _status_workspace(workspace, index), _stream(index)), "kda_page_compact")
    return table_out, refs_out, free_out, pairs, count, moved
