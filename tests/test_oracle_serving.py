"""The serving oracle against separate statements of the same definitions."""

import pytest
import torch

from oracle import latent as ol
from oracle import serving as sv


def test_chunk_is_the_expanded_form_of_its_rows():
    g = torch.Generator().manual_seed(1)
    lens_q, lens, H, size = [3, 0, 5], [20, 7, 5], 2, 4
    cache = torch.randn(12, size, 576, generator=g).double()
    table = torch.tensor([[3, 1, 0, 7, 2], [4, 5, -1, -1, -1], [9, 11, -1, -1, -1]])
    q, w = torch.randn(8, H, 192, generator=g).double(), torch.randn(H, 256, 512, generator=g).double() / 20
    rows = torch.cat([cache[table[0]].reshape(-1, 576)[:20], cache[[9, 11]].reshape(-1, 576)[:5]])
    kv = torch.einsum("jc,hdc->jhd", rows[:, :512], w)
    want = ol.latent_fwd(q, kv, rows[:, 512:], [3, 5], [20, 5])
    got = sv.latent_chunk(q, cache, table, lens, w, lens_q)
    torch.testing.assert_close(got[0], want[0], rtol=1e-12, atol=1e-13)
    torch.testing.assert_close(got[1], want[1], rtol=1e-12, atol=1e-13)
    assert (got[2] >= want[2] * (1 - 1e-9)).all()


def test_rounded_values_and_their_neighbours():
    x = torch.tensor([1.0 + 2.0 ** -8, 1.0, 1.0 + 2.0 ** -8 - 2.0 ** -30]).double()   # on a border of bf16, on a value
    mid, off = sv._rounded(x, torch.tensor([2.0 ** -13, 2.0 ** -13, 2.0 ** -13]).double(), torch.bfloat16)
    assert mid.tolist() == [1.0, 1.0, 1.0] and off.tolist() == [2.0 ** -7, 0.0, 2.0 ** -7]


@pytest.mark.parametrize("drafted", [True, False])
def test_accepted_and_drawn_tokens_have_the_targets_distribution(drafted):
    """Over a grid of both uniform numbers and all drafts, weighted by the proposer's probabilities (whole multiples of
    the grid's step, so the counts are exact)."""
    p, q, steps = [1, 0, 5, 2], [4, 1, 2, 1], 8
    probs = lambda r: torch.tensor(r).float().div(8)  # noqa: E731
    target, draft = torch.stack([probs(p), probs(p)])[None], probs(q)[None, None]
    fine = 8 * 3 * 7                                          # the rests sum to 4 eighths, and to 7, 8, 3 and 6
    count = [0.0] * 4
    for d in range(4):
        for s in range(steps):
            for t in range(fine):
                u = torch.tensor([[(s + 0.5) / steps, (t + 0.5) / fine]])
                if drafted:
                    (a, tok), = sv.verify_drafts(torch.tensor([[d]]), target, u, draft)
                else:
                    (a, tok), = sv.verify_drafts(torch.tensor([[d]]), target, u)
                first = d if a else tok[0]
                count[first] += q[d] / 8 / steps / fine
    # acceptance in steps of 1/8: min(1, p/q) is 1/4, 0, 1, 1 with the proposer's, p itself without
    for c, x in zip(count, p):
        assert abs(c - x / 8) < 1e-9


def test_drafts_end_and_ties():
    target = torch.full((1, 3, 4), 0.25)
    u = lambda *x: torch.tensor([x])  # noqa: E731
    # u = k / V exactly: the sums up to k - 1 are not above it
    for k in range(4):
        assert sv.verify_drafts(torch.tensor([[-1, 2]]), target, u(0.0, 0.0, k / 4), slack=0.0) == [(0, [k])]
    assert sv.verify_drafts(torch.tensor([[3, -1]]), target, u(0.0, 0.0, 0.75), target[:, :2]) == [(1, [2, 3])]
    assert sv.verify_drafts(torch.tensor([[3, 4]]), target, u(0.0, 0.0, 0.9), target[:, :2]) == [(1, [3])]
    assert sv.verify_drafts(torch.tensor([[0, 0]]), target, u(1.0, 0.0, 0.3), target[:, :2]) == [(0, [1])]   # p = q
    assert sv.verify_drafts(torch.tensor([[0, 0]]), target * 0, u(0.0, 0.0, 0.3)) == [(0, None)]


def test_pages_by_hand():
    table = torch.tensor([[5, 6, -1], [-1, -1, -1], [-1, -1, -1]])
    refs, free = [0] * 8, [5, 6, 3, 1, 0, 2, 4, 7]
    t, lens, refs, head, pairs = sv.page_fork(table, [6, 0, 0], [0, 0], [1, 2], refs, free, 2, 4)
    assert t.tolist() == [[5, 6, -1], [5, 3, -1], [5, 1, -1]] and lens == [6, 6, 6] and head == 4
    assert refs == [0, 0, 0, 0, 0, 2, 0, 0] and pairs == [(6, 3), (6, 1)]
    lens, refs, free, head = sv.page_free(t, lens, [0, 4, 6], refs, free, head, 4)
    assert lens == [0, 4, 6] and refs == [0, 0, 0, 0, 0, 1, 0, 0] and head == 2 and free[2:] == [3, 6, 0, 2, 4, 7]
    t, refs, free, pairs, count, moved = sv.page_compact(t, lens, refs, free, head, 4)
    assert count == 1 and pairs[0] == (5, 0) and moved == [-1, 1, -1, -1, -1, 0, -1, -1]
    assert t.tolist() == [[-1, -1, -1], [0, -1, -1], [0, 1, -1]] and refs == [1] + [0] * 7 and free == [5, 6, 2, 3, 4, 5, 6, 7]
