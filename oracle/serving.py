"""Serving over the paged latent cache from its definitions: chunks of new
tokens in 64 bits, drafts in whole numbers, pages one at a time.

TEST INFRASTRUCTURE ONLY: the oracle of ``kda_latent_chunk``,
``kda_verify_drafts``, ``kda_page_fork``, ``kda_page_free`` and
``kda_page_compact``.  Arguments are torch CPU tensors or lists; nothing here
is shared with the CUDA path.
"""

from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

from .latent import F32, KEY, LATENT, SCALE, VAL, _sees, attention


# ---------------------------------------------------------------------------
def cached_rows(cache, table, n: int, length: int) -> torch.Tensor:
    """The first `length` rows of sequence n; zeros where its page does not exist."""
    pages, size, width = cache.shape
    rows = torch.zeros(length, width, dtype=torch.float64)
    for j in range(length):
        page = int(table[n, j // size])
        if 0 <= page < pages:
            rows[j] = cache[page, j % size].double()
    return rows


def _rounded(x, spread, dtype) -> Tuple[torch.Tensor, torch.Tensor]:
    """x rounded to the type, and how far the rounding of a 32-bit sum of 512 products whose sizes add up to `spread`
    may be from it: another value where the sum's error reaches over a border."""
    if dtype is None:
        return x, torch.zeros_like(x)
    off = 512 * F32 * spread + 2 * F32 * x.abs()   # (a conversion from 64 bits goes through 32)
    low, high = (x - off).to(dtype).double(), (x + off).to(dtype).double()
    mid = x.to(dtype).double()
    return mid, torch.maximum(high - mid, mid - low)


def _as_two(x, spread, u: float, tiny: float) -> Tuple[torch.Tensor, torch.Tensor]:
    """x, and how far a sum of two numbers of a type with unit u may be from it, which a 32-bit sum was split into."""
    return x, 512 * F32 * spread + u * u * x.abs() + tiny


def latent_chunk(q, cache, table, lens: Sequence[int], w_up, lens_q: Sequence[int], scale: Optional[float] = None,
                 dtype=None, u: float = 0.0, tiny: float = 0.0, few: int = 0):
    """q [T, H, 192] (packed by lens_q).  With `dtype` the expanded values are rounded to it, and the keys, but for
    query pairs of tiles (256 rows) that see at most `few` keys, for which they are sums of two such numbers.  Returns
    (o, lse, err_o, err_lse), the errors' bounds as in ``latent.attention`` with what the expanded values may be off."""
    scale = SCALE if scale is None else scale
    q, w = q.double(), w_up.double()
    T, H, _ = q.shape
    o = torch.zeros(T, H, VAL, dtype=torch.float64)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    a = 0
    for n, (lq, lk) in enumerate(zip(lens_q, lens)):
        rows = cached_rows(cache, table, n, lk) if lq else None
        for first in range(0, lq, 256):
            pair = slice(first, min(lq, first + 256))
            at = slice(a + pair.start, a + pair.stop)
            sees = _sees(lq, lk, True)[pair]
            two = -(-max(0, min(lk, pair.stop + lk - lq)) // 128) * 128 <= few
            c, pe = rows[:, :LATENT], rows[:, LATENT:]
            for h in range(H):
                wk, wv = w[h, :KEY], w[h, KEY:]
                spread = c.abs() @ wk.abs().T
                k, ek = _as_two(c @ wk.T, spread, u, tiny) if two else _rounded(c @ wk.T, spread, dtype)
                v, ev = _rounded(c @ wv.T, c.abs() @ wv.abs().T, dtype)
                qi, k = q[at, h], torch.cat([k, pe], 1)
                # (the scores' sums are 128 products longer where the keys are two numbers)
                ro, rl, e, x = attention(qi, k, v, sees, scale, u, tiny)
                more = torch.zeros(len(qi), dtype=torch.float64)
                if lk:
                    none = torch.zeros(len(qi), lk, dtype=torch.float64)
                    more = torch.where(sees, scale * (qi[:, :KEY].abs() @ ek.T), none).amax(-1)
                    if two:
                        more = more + 128 * F32 * scale * torch.where(sees, qi.abs() @ k.abs().T, none).amax(-1)
                    p = torch.nan_to_num(torch.softmax(torch.where(sees, scale * (qi @ k.T), none - float("inf")), -1))
                    e = e + 2 * more[:, None] * (p @ v.abs()) + p @ ev
                o[at, h], lse[at, h], eo[at, h], el[at, h] = ro, rl, e, x + more
        a += lq
    return o, lse, eo, el


# ---------------------------------------------------------------------------
_UNIT = 1 << 149   # every fp32 number is a whole number of 2^-149


def _whole(row) -> List[int]:
    """Finite numbers above zero as whole numbers of 2^-149; the others, which have no weight, as 0."""
    out = []
    for x in row.float().tolist():
        if x > 0 and x != float("inf"):
            a, b = x.as_integer_ratio()
            out.append(a * (_UNIT // b))
        else:
            out.append(0)
    return out


def verify_drafts(drafts, target, uniform, draft_probs=None, slack: float = 2.0 ** -44):
    """For each sequence (accepted drafts, the tokens that may stand behind them): more than one where the border is
    within `slack` of the sum, None where nothing has weight."""
    V, out = target.shape[2], []
    for n in range(drafts.shape[0]):
        tokens, a, rejected = drafts[n].tolist(), 0, False
        for s, d in enumerate(tokens):
            if d < 0 or d >= V:
                break
            u, p = _whole(uniform[n, s:s + 1])[0], _whole(target[n, s, d:d + 1])[0]
            q = _whole(draft_probs[n, s, d:d + 1])[0] if draft_probs is not None else _UNIT
            if u * q >= p * _UNIT:
                rejected = True
                break
            a += 1
        p = _whole(target[n, a])
        r = p
        if rejected:
            if draft_probs is None:
                r = [0 if i == tokens[a] else x for i, x in enumerate(p)]
            else:
                r = [max(x - y, 0) for x, y in zip(p, _whole(draft_probs[n, a]))]
            if sum(r) == 0:
                r = p
        total = sum(r)
        if total == 0:
            out.append((a, None))
            continue
        border = _whole(uniform[n, -1:])[0] * total          # in units of 2^-298
        wide = int(slack * 2 ** 60) * total * (_UNIT >> 60)
        sums, allowed, last = 0, [], None
        for i, x in enumerate(r):
            if x == 0:
                continue
            before, sums, last = sums, sums + x, i
            if before * _UNIT <= border + wide and sums * _UNIT > border - wide:
                allowed.append(i)
        out.append((a, allowed or [last]))
    return out


# ---------------------------------------------------------------------------
def _pages(length: int, size: int) -> int:
    return -(-length // size)


def page_fork(table, lens, parents, children, refs, free, head: int, size: int, fork_lens=None):
    """Returns (table, lens, refs, head, pairs) anew."""
    table, new, refs, pairs = table.clone(), list(lens), list(refs), []
    for i, (a, c) in enumerate(zip(parents, children)):
        pair = (-1, -1)
        if c >= 0:
            length = lens[a] if fork_lens is None else fork_lens[i]
            full = length // size
            for j in range(full):
                table[c, j] = table[a, j]
                refs[int(table[a, j])] += 1
            if length % size:
                pair = (int(table[a, full]), int(free[head]))
                table[c, full] = free[head]
                head += 1
            new[c] = length
        pairs.append(pair)
    return table, new, refs, head, pairs


def page_free(table, lens, keep, refs, free, head: int, size: int):
    """Returns (lens, refs, free, head) anew."""
    refs, free, gone = list(refs), list(free), []
    for n, (length, kept) in enumerate(zip(lens, keep)):
        for j in range(_pages(kept, size), _pages(length, size)):
            page = int(table[n, j])
            if refs[page] == 0:
                gone.append(page)
            else:
                refs[page] -= 1
    for i, page in enumerate(sorted(gone)):
        free[head - len(gone) + i] = page
    return list(keep), refs, free, head - len(gone)


def page_compact(table, lens, refs, free, head: int, size: int):
    """Returns (table, refs, free, pairs, count, moved)."""
    pages = len(refs)
    there = set(free[head:])
    used = [p for p in range(pages) if p not in there]
    holes = [p for p in range(len(used)) if p in there]
    movers = [p for p in used if p >= len(used)]
    moved = [-1 if p in there else p for p in range(pages)]
    for a, b in zip(movers, holes):
        moved[a] = b
    new = [0] * pages
    for p in used:
        new[moved[p]] = refs[p]
    out = torch.full_like(table, -1)
    for n, length in enumerate(lens):
        for j in range(_pages(length, size)):
            out[n, j] = moved[int(table[n, j])]
    pairs = list(zip(movers, holes))
    rest = [len(used) + i for i in range(len(free) - head)]
    return out, new, list(free[:head]) + rest, pairs + [(-1, -1)] * (pages // 2 - len(pairs)), len(pairs), moved
