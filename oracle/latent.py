"""Latent attention, its cache and its tables from their definitions, in 64 bits.

TEST INFRASTRUCTURE ONLY: the oracle of ``kda_latent_fwd``, ``kda_latent_bwd``,
``kda_latent_decode``, ``kda_latent_append`` and ``kda_block_tables``.

One sequence and head at a time, scores written out, no tiling, no running
statistics.  Besides each result the functions return a first-order bound of
what 16-bit operands and 32-bit sums may add to it (``err``): a rounding to a
type with unit ``u`` (half its ``eps``) is off by at most ``u`` of its value.
fp16 besides has a smallest step, 2^-24: ``tiny`` is half of it (0 for bf16,
whose range is fp32's).  Arguments are torch CPU tensors; nothing here is
shared with the CUDA path.
"""

from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

PE, KEY, VAL, LATENT = 64, 128, 128, 512
SCALE = 192.0 ** -0.5
F32 = 2.0 ** -24


def _sees(lq: int, lk: int, causal: bool) -> torch.Tensor:
    sees = torch.ones(lq, lk, dtype=torch.bool)
    if causal:
        for i in range(lq):
            sees[i, max(0, i + lk - lq + 1):] = False
    return sees


def _softmax(x: torch.Tensor, sees: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Weights (zero where nothing is seen) and log-sum-exp (-inf there) of masked rows."""
    x = torch.where(sees, x, torch.full_like(x, -float("inf")))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.where(sees, p, torch.zeros_like(p)), lse


def attention(q, k, v, sees, scale: float, u: float = 0.0, tiny: float = 0.0):
    """One head: (o, lse, err_o, err_lse) of q [Lq, D], k [Lk, D], v [Lk, E]."""
    x = scale * (q @ k.T)
    p, lse = _softmax(x, sees)
    # a score is a sum of D products in 32 bits; D 2^-24 of its terms' sizes, on the row's largest
    dx = torch.zeros(q.shape[0], dtype=torch.float64)
    if k.shape[0]:
        dx = q.shape[1] * F32 * scale * torch.where(sees, q.abs() @ k.abs().T, torch.zeros_like(x)).amax(-1)
    dx = dx + 2.0 ** -20                     # exponentials and sums of the weights
    spread = p @ v.abs()
    o = p @ v
    # the weights are rounded relative to a reference at which the largest is at least 1
    err = u * o.abs() + (u + 2 * dx[:, None]) * spread + tiny * (1 + sees.double() @ v.abs())
    return o, lse, err, dx + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def latent_fwd(q, kv, k_pe, lens_q: Sequence[int], lens_k: Sequence[int], causal: bool = True,
               scale: Optional[float] = None, u: float = 0.0, tiny: float = 0.0):
    """Packed rows q [Tq, H, 192], kv [Tk, H, 256], k_pe [Tk, 64].  Returns (o, lse, err_o, err_lse)."""
    scale = SCALE if scale is None else scale
    q, kv, k_pe = q.double(), kv.double(), k_pe.double()
    tq, H, _ = q.shape
    o = torch.zeros(tq, H, VAL, dtype=torch.float64)
    lse = torch.full((tq, H), -float("inf"), dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        sees = _sees(lq, lk, causal)
        for h in range(H):
            k = torch.cat([kv[b:b + lk, h, :KEY], k_pe[b:b + lk]], -1)
            r = attention(q[a:a + lq, h], k, kv[b:b + lk, h, KEY:], sees, scale, u, tiny)
            o[a:a + lq, h], lse[a:a + lq, h], eo[a:a + lq, h], el[a:a + lq, h] = r
        a, b = a + lq, b + lk
    return o, lse, eo, el


def latent_bwd(q, kv, k_pe, do, lens_q: Sequence[int], lens_k: Sequence[int], causal: bool = True,
               scale: Optional[float] = None, u: float = 0.0, tiny: float = 0.0):
    """Gradients of sum <do, o> by the formulas.  Returns (dq, dkv, dk_pe, err_dq, err_dkv, err_dk_pe)."""
    scale = SCALE if scale is None else scale
    q, kv, k_pe, do = q.double(), kv.double(), k_pe.double(), do.double()
    dq, dkv, dpe = torch.zeros_like(q), torch.zeros_like(kv), torch.zeros_like(k_pe)
    eq, ekv, epe = torch.zeros_like(q), torch.zeros_like(kv), torch.zeros_like(k_pe)
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        sees = _sees(lq, lk, causal)
        for h in range(q.shape[1]):
            qi, di = q[a:a + lq, h], do[a:a + lq, h]
            k = torch.cat([kv[b:b + lk, h, :KEY], k_pe[b:b + lk]], -1)
            v = kv[b:b + lk, h, KEY:]
            p, _ = _softmax(scale * (qi @ k.T), sees)
            o = p @ v
            big = torch.where(sees, qi.abs() @ k.abs().T, torch.zeros_like(p))
            dx = (192 * F32 * scale * big.amax(-1) if lk else torch.zeros(lq, dtype=torch.float64)) + 2.0 ** -20
            w = p * (di @ v.T - (di * o).sum(-1, keepdim=True))
            # each weight is off by 2 dx of itself; its row's D by what o was; do . v by its 32-bit sum; w is rounded
            d_o = u * o.abs() + (u + 2 * dx[:, None]) * (p @ v.abs()) + tiny * (1 + sees.double() @ v.abs())
            ew = (u + 2 * dx[:, None]) * w.abs() + p * ((di.abs() * d_o).sum(-1, keepdim=True) + 128 * F32 * (di.abs() @ v.abs().T + (di * o).abs().sum(-1, keepdim=True))) + tiny * sees
            dq[a:a + lq, h] = scale * (w @ k)
            dk = scale * (w.T @ qi)
            dv = p.T @ di
            eq[a:a + lq, h] = u * dq[a:a + lq, h].abs() + tiny + scale * (ew @ k.abs())
            ek = scale * (ew.T @ qi.abs())
            dkv[b:b + lk, h] = torch.cat([dk[:, :KEY], dv], -1)
            ev = (p * (u + 2 * dx[:, None]) + tiny * sees).T @ di.abs()
            ekv[b:b + lk, h] = u * dkv[b:b + lk, h].abs() + tiny + torch.cat([ek[:, :KEY], ev], -1)
            dpe[b:b + lk] += dk[:, KEY:]
            epe[b:b + lk] += ek[:, KEY:]
        a, b = a + lq, b + lk
    return dq, dkv, dpe, eq, ekv, epe + u * dpe.abs() + tiny


def latent_bwd_norms(q, kv, k_pe, do, lens_q: Sequence[int], lens_k: Sequence[int], scale: Optional[float] = None,
                     u: float = 0.0, tiny: float = 0.0):
    """Causal gradients whose errors are bounded in the Frobenius norm, a sequence and head at a time (the elementwise
    bounds of latent_bwd add up absolute values and are some sqrt(L) wider, and they admit half a smallest step in
    every weight).  o, lse: the exact ones, o rounded to the tensors' type, are what the backward is given.  Returns
    (o, lse, [per sequence and head: dict of name -> (rows, head, channels, exact gradient, bound)]) with the names dq,
    dk, dv; the shared key's gradient is summed over the heads, name dpe, head None.

    dS = p (dP - D) is off by twice the scores' error and by one rounding of itself (u; its smallest step must not
    count), by the 32-bit sums of dP, and by D's change with o's rounding.  A product with a matrix M then is off by at
    most |error|_F |M|_2, by its own 32-bit sums (at most L steps of partial sums of that size) and by the result's
    rounding."""
    scale = SCALE if scale is None else scale
    typed = q.dtype
    q, kv, k_pe, do = q.double(), kv.double(), k_pe.double(), do.double()
    o, lse, _, _ = latent_fwd(q, kv, k_pe, lens_q, lens_k, True, scale)
    given = o.to(typed).double()
    norm = lambda x: float(torch.linalg.matrix_norm(x)) if x.numel() else 0.0  # noqa: E731
    spectral = lambda x: float(torch.linalg.matrix_norm(x, 2)) if x.numel() else 0.0  # noqa: E731
    rounded = lambda x: norm((u * x.abs()).clamp(min=tiny))  # noqa: E731
    out, a, b = [], 0, 0
    for lq, lk in zip(lens_q, lens_k):
        sees, dpe, epe = _sees(lq, lk, True), torch.zeros(lk, PE, dtype=torch.float64), 0.0
        for h in range(q.shape[1]):
            rq, rk = slice(a, a + lq), slice(b, b + lk)
            qi, di, v = q[rq, h], do[rq, h], kv[rk, h, KEY:]
            k = torch.cat([kv[rk, h, :KEY], k_pe[rk]], -1)
            p, _ = _softmax(scale * (qi @ k.T), sees)
            ds = p * (di @ v.T - (di * o[rq, h]).sum(-1, keepdim=True))
            big = torch.where(sees, qi.abs() @ k.abs().T, torch.zeros_like(p)).amax(-1)
            dx = 192 * F32 * scale * big + 2.0 ** -20 + F32 * lse[rq, h].abs().nan_to_num(posinf=0.0)
            d_d = (di.abs() * (given[rq, h] - o[rq, h]).abs()).sum(-1, keepdim=True)
            sums = 128 * F32 * (di.abs() @ v.abs().T + (di * o[rq, h]).abs().sum(-1, keepdim=True))
            e_ds = norm((u + 2 * dx[:, None]) * ds.abs() + p * sums)
            steps = F32 * max(lq, lk) * norm(ds)
            dq, dk, dv = scale * (ds @ k), scale * (ds.T @ qi), p.T @ di
            e_q = scale * ((e_ds + steps) * spectral(k) + norm(d_d * (p @ k)))
            e_k = scale * ((e_ds + steps) * spectral(qi) + norm(p.T @ (d_d * qi.abs())))
            # (a weight carries 2^8 in the tensors' type: half of its smallest step is tiny 2^-8)
            e_v = (norm((u + 2 * dx[:, None]) * p) + F32 * lq * norm(p) + tiny * 2.0 ** -8 * float(sees.sum()) ** 0.5) * spectral(di)
            out.append(dict(dq=(rq, h, slice(0, 192), dq, e_q + rounded(dq)),
                            dk=(rk, h, slice(0, KEY), dk[:, :KEY], e_k + rounded(dk[:, :KEY])),
                            dv=(rk, h, slice(KEY, KEY + VAL), dv, e_v + rounded(dv))))
            dpe += dk[:, KEY:]
            epe += e_k
        out.append(dict(dpe=(slice(b, b + lk), None, slice(0, PE), dpe, epe + rounded(dpe))))
        a, b = a + lq, b + lk
    return o, lse, out


def latent_decode(q, cache, table, lens, scale: Optional[float] = None, u: float = 0.0, tiny: float = 0.0):
    """q [N, S, H, 576], cache [pages, page_size, 576], table [N, W], lens [N].  Rows on a page that does not
    exist are masked, lengths are clipped to the table.  Returns (o, lse, err_o, err_lse)."""
    scale = SCALE if scale is None else scale
    n, s, H, _ = q.shape
    pages, ps, _ = cache.shape
    o = torch.zeros(n, s, H, LATENT, dtype=torch.float64)
    lse = torch.full((n, s, H), -float("inf"), dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(n):
        length = min(max(int(lens[i]), 0), table.shape[1] * ps)
        ids = [int(table[i, j // ps]) for j in range(length)]
        there = torch.tensor([0 <= page < pages for page in ids], dtype=torch.bool)
        rows = torch.stack([cache[page, j % ps].double() if 0 <= page < pages else torch.zeros(576, dtype=torch.float64)
                            for j, page in enumerate(ids)]) if length else torch.zeros(0, 576, dtype=torch.float64)
        for t in range(s):
            seen = max(0, length - s + 1 + t)
            sees = (torch.arange(length) < seen) & there if length else torch.zeros(0, dtype=torch.bool)
            r = attention(q[i, t].double(), rows, rows[:, :LATENT], sees[None].expand(H, -1), scale, u)
            o[i, t], lse[i, t], eo[i, t], el[i, t] = r
    return o, lse, eo, el


def latent_append(rows, slots, cache, weight=None, eps: float = 1e-6) -> torch.Tensor:
    """The cache in 64 bits after the rows are written."""
    out = cache.double().clone()
    flat = out.view(-1, out.shape[-1])
    for row, slot in zip(rows.double(), slots.tolist()):
        if 0 <= slot < flat.shape[0]:
            row = row.clone()
            if weight is not None:
                row[:LATENT] *= (row[:LATENT].square().mean() + eps) ** -0.5 * weight.double()
            flat[slot] = row
    return out


def block_tables(lens: List[int], new: List[int], table: List[List[int]], free: List[int], head: int, page_size: int,
                 num_tokens: int):
    """One token after another.  Returns (slots, cu, lens_out, head_out, table)."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    slots, cu, out, at = [], [0], [], head
    for n, (a, b) in enumerate(zip(lens, new)):
        a, b = max(a, 0), max(b, 0)
        held = -(-a // page_size)
        for pos in range(a, a + b):
            cell = pos // page_size
            if cell >= width:
                slots.append(-1)
                continue
            if cell >= held and (pos % page_size == 0 or pos == a):
                table[n][cell] = free[at] if 0 <= at < len(free) else -1
                at += 1
            page = table[n][cell]
            slots.append(-1 if page < 0 else page * page_size + pos % page_size)
        cu.append(cu[-1] + b)
        out.append(a + b)
    slots = (slots + [-1] * num_tokens)[:num_tokens]
    return slots, cu, out, min(at, len(free)), table
