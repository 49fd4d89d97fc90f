"""Serving over the paged cache at the edges of its types, sizes and threads."""

import threading
from fractions import Fraction

import pytest
import torch

from oracle import serving as sv
from test_serving_gpu import (BF, F32, FEW, FP, check_drafts, chunk_inputs, draft_inputs, i32, lengths, pages, pool_state, run_chunk,
                              status, verify)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# keys past the largest number
@pytest.mark.parametrize("dtype,row,ups", [(FP, 300.0, (200.0, 300.0)), (BF, 1e20, (1e10, 1e20))])
def test_chunk_keys_past_the_largest_number_are_infinite(dtype, row, ups):
    """One channel of one cached row's key: the largest numbers, and past them.  Where queries meet it with the other
    sign its score is that far below the others, or minus infinity: the same bits, whether the keys are two numbers
    (up to FEW) or one.  With its own sign an infinite key leaves no number."""
    lens_q, lens, H, at = [20, 20, 300], [FEW[dtype] - 56, FEW[dtype] + 130, FEW[dtype] + 40], 2, (7, 100, 60)
    q, cache, table, w = chunk_inputs(lens_q, lens, H, 16, dtype, seed=3)
    cache[..., 0], w[:, :, 0] = 0, 0
    for n, j in enumerate(at):
        cache[table[n, j // 16], j % 16, 0] = row
    meets = torch.cat([j <= torch.arange(lq) + lk - lq for j, lq, lk in zip(at, lens_q, lens)]).cuda()
    assert meets[:40].all() and 200 < meets[40:].sum()
    q[..., 5] = -q[..., 5].abs().clamp(min=0.25)
    got = []
    for up in ups:
        w[:, 5, 0] = up
        got.append(run_chunk(q, cache, table, lens, w, lens_q))
    for a, b in zip(*got):
        assert not torch.isnan(a).any() and torch.equal(a, b)
    q[..., 5] = q[..., 5].abs()
    o, lse = run_chunk(q, cache, table, lens, w, lens_q)
    assert torch.isnan(o[meets]).all() and torch.isnan(lse[meets]).all() and not torch.isnan(lse[~meets]).any()
    q[::2, :, 5] *= -1                                   # rows of either sign in one tile
    o, lse = run_chunk(q, cache, table, lens, w, lens_q)
    assert torch.equal(o[::2], got[1][0][::2]) and torch.equal(lse[::2], got[1][1][::2]) and torch.isnan(o[1::2][meets[1::2]]).all()


# ---------------------------------------------------------------------------
# threads
def test_pools_of_different_size_are_compacted_by_two_threads():
    from chunked_gated_delta_kda_gb300 import pages
    sizes, failed, got = (512, 1 << 20), [], {}

    def work(size):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                held = size // 2
                order = torch.arange(size, dtype=torch.int32, device="cuda").flip(0)
                args = order[None, :held].contiguous(), i32([held]), torch.zeros_like(order), order, i32([held]), 1
                torch.cuda.current_stream().synchronize()
                for _ in range(3000):
                    out = pages.page_compact(*args)
                torch.cuda.current_stream().synchronize()
                got[size] = [x.cpu() for x in out]
        except Exception as e:                           # (of a thread: told below)
            failed.append((size, e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(size,)) for size in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for size in sizes:
        table, _, free, pairs, count, moved = got[size]
        held = size // 2
        assert count.item() == held and torch.equal(table[0].sort().values, torch.arange(held, dtype=torch.int32))
        assert torch.equal(free[held:], torch.arange(held, size, dtype=torch.int32)) and torch.equal(moved[pairs[:, 0].long()], pairs[:, 1])


# ---------------------------------------------------------------------------
# long rows of probabilities
def halves_row(V, numbers, dtype):
    """[1, 1, V], the first half of it one number, the second half another."""
    row = torch.full((1, 1, V), numbers[0], dtype=dtype, device="cuda")
    row[..., V // 2:] = numbers[1]
    return row


def check_halves(tokens, u, V, ends, weights, slack):
    """Drawn tokens of a row whose weights are 0, then weights[0] from ends[0] on and weights[1] from V / 2 on: each
    one's sums, exact, enclose its border within slack of the total."""
    a, b = (Fraction(w) for w in weights)
    upto = lambda i: a * (min(i, V // 2) - ends) + b * max(0, i - V // 2)  # noqa: E731  (weight of the tokens before i)
    total = upto(V)
    for token, x in zip(tokens.tolist(), u.tolist()):
        assert ends <= token < V
        border, off = Fraction(x) * total, Fraction(slack) * total
        assert upto(token) <= border + off and upto(token + 1) > border - off, (token, float((upto(token + 1) - border) / total))


ROWS = 153   # as many as leave a sequence one CTA, whose sums are the longest


@pytest.mark.parametrize("V,slack", [(1 << 18, 2.0 ** -40), (1 << 22, 2.0 ** -33), (1 << 28, 2.0 ** -31)])
def test_drafts_of_long_rows(V, slack):
    """A number whose sums round the same way for many steps, beside one that is summed exactly; all sequences read one
    row."""
    weights = 1.0, torch.tensor(1.74220228).item()
    target = halves_row(V, weights, F32).expand(ROWS, 1, V)
    u = torch.rand(ROWS, 1, generator=torch.Generator().manual_seed(V))
    out, n = verify(torch.zeros(ROWS, 0, dtype=torch.int64, device="cuda"), target, u.cuda())
    assert (n == 1).all()
    check_halves(out[:, 0].cpu(), u[:, 0], V, 0, weights, slack)
    one = halves_row(V, weights, F32)          # and by eight
    out, _ = verify(torch.zeros(1, 0, dtype=torch.int64, device="cuda"), one, u[:1].cuda())
    check_halves(out[:, 0].cpu(), u[:1, 0], V, 0, weights, slack)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_drafts_of_long_rows_with_a_proposers(dtype):
    """max(p - q, 0) of two rows; the draft has no probability and is rejected."""
    V, S = 1 << 26, 1
    p, q = halves_row(V, (1.5, 1.7421875), dtype), halves_row(V, (0.5, 0.0145111083984375), dtype)
    weights = [float(p[0, 0, i].double() - q[0, 0, i].double()) for i in (0, V - 1)]
    p[..., 0] = 0
    u = torch.rand(ROWS, 2, generator=torch.Generator().manual_seed(5))
    out, n = verify(torch.zeros(ROWS, S, dtype=torch.int64, device="cuda"), p.expand(ROWS, 2, V), u.cuda(), q.expand(ROWS, 1, V))
    assert (n == 1).all() and (out[:, 1] == -1).all()
    check_halves(out[:, 0].cpu(), u[:, 1], V, 1, weights, 2.0 ** -31)


@pytest.mark.parametrize("V,dtype", [(262144, F32), (262147, BF), (1000003, FP)])
def test_drafts_of_large_vocabularies(V, dtype):
    check_drafts(*draft_inputs(2, 1, V, dtype, seed=V))


# ---------------------------------------------------------------------------
# pages
@pytest.mark.parametrize("n,width", [(255, 512), (256, 512), (257, 512), (4, 40000)])
def test_rejected_drafts_in_tables_around_the_border(n, width):
    """Up to seven tokens back, in tables of as many cells as one cluster gives back, and of more."""
    lens = lengths(n, 16 * width, n)
    table, refs, free, head = pool_state(lens, 16, 64, n, 1, width)
    keep = [max(0, l - (i * 5) % 8) for i, l in enumerate(lens)]
    f = i32(free)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    got = pages().page_free(table.cuda(), i32(lens), i32(keep), i32(refs), f, i32([head]), 16, workspace=ws)
    wl, wr, wf, wh = sv.page_free(table, lens, keep, refs, free, head, 16)
    assert status(ws) == 0 and got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh and f.tolist() == wf


def test_lengths_past_the_table_are_clipped_when_pages_go_back():
    """A row of 1000 tokens in a table of three pages of four gives back three."""
    table = torch.tensor([[4, 5, 6], [7, -1, -1]], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    shared = [0, 0, 0, 0, 1, 0, 0, 0]
    for keep, listed, head, refs in ((0, [9, 4, 5, 6], 1, [0] * 8), (5, [9, 0, 4, 6], 3, shared), (12, [9, 0, 4, 5], 4, shared)):
        free = i32([9, 0, 4, 5, 0, 1, 2, 3])
        lens, r, h = pages().page_free(table, i32([1000, 4]), i32([keep, 4]), i32(refs), free, i32([4]), 4, workspace=ws)
        assert status(ws) == 8 and lens.tolist() == [keep, 4] and r.tolist() == refs and h.tolist() == [head]
        assert free.tolist() == listed + [0, 1, 2, 3]


@pytest.mark.parametrize("listed", [-7, -1, 8, 1 << 30])
def test_a_listed_page_that_is_none_becomes_none_in_a_forks_table(listed):
    table = torch.tensor([[4, 5, 6], [-1, -1, -1], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens, refs, head, pairs = pages().page_fork(table, i32([10, 0, 0]), i32([0, 0]), i32([1, 2]), i32([0] * 8), i32([4, 5, 6, listed, 3]),
                                                i32([3]), 4, workspace=ws)
    assert status(ws) == 8 and table.tolist() == [[4, 5, 6], [4, 5, -1], [4, 5, 3]] and pairs.tolist() == [[-1, -1], [6, 3]]
    assert lens.tolist() == [10, 10, 10] and refs.tolist() == [0, 0, 0, 0, 2, 2, 0, 0] and head.tolist() == [5]


@pytest.mark.parametrize("P", [2 ** 20, 2 ** 20 + 1, 2 ** 20 + 300])
def test_owners_and_tables_move_with_their_pages(P):
    """Several rows, some shorter than the table, that share pages: owners, tables and numbers as the definition gives
    them, in pools on either side of what fits as bits."""
    g = torch.Generator().manual_seed(P)
    lens = [0, 3, 5000, 4999, 1, 700, 5000 - 64, 16]
    need = [-(-n // 2) for n in lens]
    width, used = max(need) + 2, sum(need)
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.randint(-3, P + 3, (len(lens), width), generator=g).to(torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    refs = torch.zeros(P, dtype=torch.int32)
    refs[order[:used].long()] = torch.randint(0, 1000, (used,), generator=g).to(torch.int32)
    got = [x.cpu() for x in pages().page_compact(table.cuda(), i32(lens), refs.cuda(), order.cuda(), i32([used]), 2)]
    free = torch.zeros(P, dtype=torch.bool)
    free[order[used:].long()] = True
    holes, movers = free[:used].nonzero()[:, 0], (~free[used:]).nonzero()[:, 0] + used
    moved = torch.where(free, -1, torch.arange(P)).to(torch.int32)
    moved[movers] = holes.to(torch.int32)
    new = torch.zeros(P, dtype=torch.int32)
    new[moved[~free].long()] = refs[~free]
    out = torch.full_like(table, -1)
    for i, n in enumerate(need):
        out[i, :n] = moved[table[i, :n].long()]
    assert torch.equal(got[0], out) and torch.equal(got[1], new) and torch.equal(got[5], moved)
    assert torch.equal(got[2], torch.cat([order[:used], torch.arange(used, P, dtype=torch.int32)]))
    k = len(holes)
    assert got[4].item() == k and (got[3][k:] == -1).all() and torch.equal(got[3][:k], torch.stack([movers, holes], 1).to(torch.int32))


# ---------------------------------------------------------------------------
# together
def test_drafts_leave_greedy_decoding_as_it_is_past_the_border_of_few_keys():
    """A prompt that ends in front of 2048 rows, where keys are two numbers, and goes on behind them; and a longer one."""
    from chunked_gated_delta_kda_gb300.latent_serving import Decoder
    g = torch.Generator(device="cuda").manual_seed(9)
    lens = [2040, 2300]
    prompt = torch.randint(0, 50, (sum(lens),), generator=g, device="cuda")
    plain, quick = (Decoder(50, 256, 4, 2, pages=320, width=160, page_size=16, temper=1e4, seed=2) for _ in range(2))
    u = lambda s: torch.rand(2, s, generator=g, device="cuda")  # noqa: E731
    first = plain.start(prompt, i32(lens), u(1)[:, 0])
    assert torch.equal(first, quick.start(prompt, i32(lens), u(1)[:, 0]))
    want = [first]
    for _ in range(20):
        want.append(plain.step(want[-1], first.new_empty(2, 0), u(1))[0][:, 0])
    want = torch.stack(want, 1).tolist()
    texts, steps = [[t] for t in first.tolist()], 0
    while min(len(t) for t in texts) < 21:
        guess = []
        for i, t in enumerate(texts):                    # right up to a place that moves from step to step
            right = (want[i] + [0] * 9)[len(t):len(t) + 3]
            guess.append([r if k < (steps + i) % 4 else (r + 1) % 50 for k, r in enumerate(right)])
        out, count = quick.step(torch.tensor([t[-1] for t in texts], device="cuda"), torch.tensor(guess, device="cuda"), u(4))
        for t, row, c in zip(texts, out.tolist(), count.tolist()):
            t += row[:c]
        steps += 1
    for i in range(2):
        assert texts[i][:21] == want[i]
    assert steps < 20 and quick.layer.lens[0] > 2048
