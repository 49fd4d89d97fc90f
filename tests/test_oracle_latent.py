"""Pins of the latent-attention oracle (CPU): against autograd and central
differences of a separately written forward, against the identity between the
expanded and the absorbed form, and by hand for the tables."""

import numpy as np
import pytest
import torch

from oracle import latent as ol


def inputs(lens_q, lens_k, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(sum(lens_q), H, 192), r(sum(lens_k), H, 256), r(sum(lens_k), 64), r(sum(lens_q), H, 128)


def objective(q, kv, pe, do, lens_q, lens_k, causal):
    """sum <do, o>, written with explicit loops over rows."""
    total, a, b = torch.zeros((), dtype=torch.float64), 0, 0
    for lq, lk in zip(lens_q, lens_k):
        for h in range(q.shape[1]):
            for i in range(lq):
                n = max(0, min(lk, i + lk - lq + 1)) if causal else lk
                if n == 0:
                    continue
                x = (kv[b:b + n, h, :128] @ q[a + i, h, :128] + pe[b:b + n] @ q[a + i, h, 128:]) / 192 ** 0.5
                e = torch.exp(x - x.max())
                total = total + (do[a + i, h] * (e @ kv[b:b + n, h, 128:]) / e.sum()).sum()
        a, b = a + lq, b + lk
    return total


@pytest.mark.parametrize("lens_q,lens_k,causal", [([5], [5], True), ([3, 4], [7, 2], True), ([2, 3], [4, 0], False)])
def test_gradients_match_autograd_and_differences(lens_q, lens_k, causal):
    q, kv, pe, do = inputs(lens_q, lens_k, 2)
    leaves = [t.clone().requires_grad_() for t in (q, kv, pe)]
    objective(*leaves, do, lens_q, lens_k, causal).backward()
    got = ol.latent_bwd(q, kv, pe, do, lens_q, lens_k, causal)
    o = ol.latent_fwd(q, kv, pe, lens_q, lens_k, causal)[0]
    assert abs((o * do).sum() - objective(q, kv, pe, do, lens_q, lens_k, causal)) < 1e-11
    for leaf, grad in zip(leaves, got[:3]):
        assert (leaf.grad - grad).abs().max() < 1e-12
    for k in range(3):                       # a direction each: two steps, extrapolated
        d = torch.randn(got[k].shape, generator=torch.Generator().manual_seed(k), dtype=torch.float64)

        def at(t):
            args = [q, kv, pe]
            args[k] = args[k] + t * d
            return ((ol.latent_fwd(*args, lens_q, lens_k, causal)[0]) * do).sum()

        diff = [(at(s) - at(-s)) / (2 * s) for s in (2.0 ** -9, 2.0 ** -10)]
        assert abs((4 * diff[1] - diff[0]) / 3 - (got[k] * d).sum()) < 1e-8


def test_rows_without_keys():
    q, kv, pe, do = inputs([4], [2], 1)
    o, lse, _, _ = ol.latent_fwd(q, kv, pe, [4], [2], True)
    assert (o[:2] == 0).all() and torch.isinf(lse[:2]).all() and torch.isfinite(lse[2:]).all()
    assert torch.allclose(o[2], kv[0, :, 128:]) and (ol.latent_bwd(q, kv, pe, do, [4], [2], True)[0][:2] == 0).all()


def test_absorbed_is_the_expanded_form():
    """q . (W c) = (W^T q) . c and sum p (U c) = U sum p c, over a paged cache with a rotated page order."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    L, H, ps = 37, 2, 16
    c, pe, wk, wv, q = r(L, 512) / 8, r(L, 64), r(H, 128, 512) / 16, r(H, 128, 512) / 16, r(3, H, 192)
    kv = torch.cat([torch.einsum("hdc,tc->thd", wk, c), torch.einsum("hdc,tc->thd", wv, c)], -1)
    o, lse, _, _ = ol.latent_fwd(q, kv, pe, [3], [L], True)
    cache = torch.full((5, ps, 576), float("nan"), dtype=torch.float64)
    table = torch.tensor([[4, 0, 2, -1]])
    for t in range(L):
        cache[table[0, t // ps], t % ps] = torch.cat([c[t], pe[t]])
    qa = torch.cat([torch.einsum("thd,hdc->thc", q[..., :128], wk), q[..., 128:]], -1)
    oa, la, _, _ = ol.latent_decode(qa[None], cache, table, torch.tensor([L]))
    assert torch.allclose(torch.einsum("thc,hdc->thd", oa[0], wv), o, atol=1e-12) and torch.allclose(la[0], lse, atol=1e-12)


def test_decode_masks_missing_pages_and_clips_lengths():
    g = torch.Generator().manual_seed(4)
    cache = torch.randn(3, 16, 576, generator=g, dtype=torch.float64)
    q = torch.randn(2, 1, 1, 576, generator=g, dtype=torch.float64)
    o, lse, _, _ = ol.latent_decode(q, cache, torch.tensor([[0, 9], [1, 2]]), torch.tensor([32, 99]))
    one = ol.latent_decode(q[:1], cache, torch.tensor([[0]]), torch.tensor([16]))
    two = ol.latent_decode(q[1:], cache, torch.tensor([[1, 2]]), torch.tensor([32]))
    assert torch.equal(o[0], one[0][0]) and torch.equal(o[1], two[0][0]) and torch.equal(lse[1], two[1][0])
    o, lse, _, _ = ol.latent_decode(q, cache, torch.tensor([[0], [1]]), torch.tensor([0, -3]))
    assert (o == 0).all() and torch.isinf(lse).all()


def test_append():
    g = torch.Generator().manual_seed(5)
    rows, cache, w = torch.randn(3, 576, generator=g), torch.zeros(2, 4, 576), torch.rand(512, generator=g)
    out = ol.latent_append(rows, torch.tensor([7, -1, 2]), cache, w)
    x = rows[0, :512].double().numpy()
    assert np.allclose(out[1, 3, :512].numpy(), x / np.sqrt(np.mean(x * x) + 1e-6) * w.double().numpy(), atol=1e-14)
    assert torch.equal(out[1, 3, 512:], rows[0, 512:].double()) and out[0, 2].abs().sum() > 0
    assert out[0, 0].abs().sum() == 0 and torch.equal(ol.latent_append(rows, torch.tensor([7, -1, 2]), cache)[0, 2], rows[2].double())


def test_block_tables_by_hand():
    # sequence 0 holds 3 rows on page 5, gets 3: one stays there, two go to a new page; 1 gets nothing; 2 is new
    slots, cu, out, head, table = ol.block_tables([3, 4, 0], [3, 0, 1], [[5, -1], [6, -1], [-1, -1]], [9, 8, 7], 1, 4, 6)
    assert slots == [23, 32, 33, 28, -1, -1] and cu == [0, 3, 3, 4] and out == [6, 4, 1] and head == 3
    assert table == [[5, 8], [6, -1], [7, -1]]
    # too few pages, and a table too narrow
    slots, _, _, head, table = ol.block_tables([0], [9], [[-1, -1]], [3], 0, 4, 9)
    assert slots == [12, 13, 14, 15, -1, -1, -1, -1, -1] and table == [[3, -1]] and head == 1
