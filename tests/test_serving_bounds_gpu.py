"""Serving over the paged cache at the edges of its types, sizes and threads."""

import threading

import pytest
import torch

from test_serving_gpu import BF, FEW, FP, chunk_inputs, i32, run_chunk

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
