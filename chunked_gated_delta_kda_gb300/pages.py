"""Pages that several requests own (argument marshalling only).

Beside ``latent.block_tables``, which takes pages from the free list:

``page_fork``     requests that go on from another one's tokens share its pages,
``page_copy``     copies pages in the caches of all layers (or in pools of states),
``page_free``     gives back the pages behind the tokens that a request keeps,
``page_compact``  brings the pages in use onto the lowest numbers.

``refs`` (int32, a number for each page) is how many owners a page has beside
its first, so pages that ``block_tables`` takes need no entry.  Every step runs
in the kernels of ``libkda.so`` (``include/kda.h`` has the contract);
``csrc/kda_marshal.cpp`` checks the tensors, allocates outputs on their device
and calls it on torch's current stream, and what it refuses is explained here.
If the library is missing, every call raises: there is no fallback path.
"""

from __future__ import annotations

from typing import Optional, Sequence, Tuple, Union

import torch

from .binding import KdaError, load_marshal
from .latent import _check, _check_int, _same_device, _status_workspace

_I32 = torch.int32


def _explain(name, status, block_table, seq_lens, refs, free_pages, free_head, page_size, in_place, workspace, **more):
    """Raises what a table function did not go through for: the C entry's status, or what is wrong with an argument.
    ``more``: tensors of seq_lens' length, or with a name that ends in ``s_`` of one length of their own."""
    if status is not None:
        raise KdaError(status, name)
    _check_int("page_size", page_size)
    if page_size < 1:
        raise ValueError(f"page_size must be positive, got {page_size}")
    _check("block_table", block_table, _I32, (None, None))
    _check("seq_lens", seq_lens, _I32, (block_table.shape[0],))
    _check("refs", refs, _I32, (None,))
    _check("free_pages", free_pages, _I32, (None,))
    _check("free_head", free_head, _I32, (1,))
    others = {key: t for key, t in more.items() if key[-1] == "_"}
    for key, t in more.items():
        _check(key.rstrip("_"), t, _I32, (None,) if key in others else (block_table.shape[0],))
    if len({t.shape for t in others.values()}) > 1:
        raise ValueError(f"{', '.join(k.rstrip('_') for k in others)} must be of one length, got "
                         f"{[t.shape[0] for t in others.values()]}")
    for key, t in (("block_table", block_table), ("refs", refs), ("free_pages", free_pages), *more.items()):
        for size in t.shape:
            _check_int(f"a size of {key.rstrip('_')}", size)
    _same_device(seq_lens.get_device(), block_table, refs, free_pages, free_head, *more.values())
    if not dict(block_table=block_table, free_pages=free_pages).get(in_place, seq_lens[:0]).is_contiguous():
        raise ValueError(f"{in_place} must be contiguous")
    _status_workspace(workspace, seq_lens.get_device())
    raise ValueError(f"{name}: page_size must be a whole number, got {page_size!r}")


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
    out = load_marshal().page_fork(block_table, seq_lens, parents, children, refs, free_pages, free_head, page_size, fork_lens,
                                   workspace)
    if type(out) is not tuple:
        _explain("kda_page_fork", out, block_table, seq_lens, refs, free_pages, free_head, page_size, "block_table", workspace,
                 parents_=parents, children_=children, **({} if fork_lens is None else dict(fork_lens_=fork_lens)))
    return out


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
    out = load_marshal().page_copy(pools, pairs, count, workspace)
    if type(out) is tuple:
        return pools
    if out is not None:
        raise KdaError(out, "kda_page_copy")
    if not isinstance(pools, (torch.Tensor, list, tuple)):
        raise TypeError("pools must be a torch.Tensor or a list of them")
    several = (pools,) if isinstance(pools, torch.Tensor) else pools
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
    _check("pairs", pairs, _I32, (None, 2))
    if count is not None:
        _check("count", count, _I32, (1,))
    _check_int("a size of pairs", pairs.shape[0])
    _check_int("a size of pools", first.shape[0])
    _same_device(first.get_device(), pairs, count, *several)
    _status_workspace(workspace, first.get_device())
    raise ValueError("pools must have pages of a multiple of 16 bytes that start on 16 bytes, got "
                     f"{first.shape[0]} in {first.numel() * first.element_size()} bytes")


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
    out = load_marshal().page_free(block_table, seq_lens, keep_lens, refs, free_pages, free_head, page_size, workspace)
    if type(out) is not tuple:
        _explain("kda_page_free", out, block_table, seq_lens, refs, free_pages, free_head, page_size, "free_pages", workspace,
                 keep_lens=keep_lens)
    return out


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
    out = load_marshal().page_compact(block_table, seq_lens, refs, free_pages, free_head, page_size, workspace)
    if type(out) is not tuple:
        _explain("kda_page_compact", out, block_table, seq_lens, refs, free_pages, free_head, page_size, None, workspace)
    return out
