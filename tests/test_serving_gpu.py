"""Chunks over the paged cache, drafts and pages on the GPU against the oracle
(``oracle.serving``): floats element by element within its bounds, whole
numbers exactly."""

import pytest
import torch

from oracle import serving as sv

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, FP: 2.0 ** -11}
TINY = {BF: 0.0, FP: 2.0 ** -25}
FEW = {BF: 2048, FP: 256}


def latent():
    from chunked_gated_delta_kda_gb300 import latent
    return latent


def pages():
    from chunked_gated_delta_kda_gb300 import pages
    return pages


def verify(*a, **kw):
    from chunked_gated_delta_kda_gb300 import drafts
    return drafts.verify_drafts(*a, **kw)


def status(ws):
    from chunked_gated_delta_kda_gb300 import binding
    return binding.get_status(ws)


def near(got, want, err, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    inf = torch.isinf(want)
    assert torch.equal(inf, torch.isinf(got)) and torch.equal(want[inf], got[inf]), what
    off = ((got - want).abs() - err)[~inf]
    assert torch.isfinite(got[~inf]).all() and (off <= 0).all(), (what, off.max().item())


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu(lens):
    return i32([sum(lens[:i]) for i in range(len(lens) + 1)])


# ---------------------------------------------------------------------------
# chunk
def paged(lens, page, dtype, seed, fill=0.0, spare=3, width=None):
    """Cache whose rows past each sequence's end, and unused pages, are `fill`; tables with -7 behind the pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-l // page) for l in lens]
    order = torch.randperm(sum(need) + spare, generator=g)
    cache = torch.full((sum(need) + spare, page, 576), fill, dtype=dtype)
    table = torch.full((len(lens), width or max(1, max(need))), -7, dtype=torch.int32)
    at = 0
    for i, l in enumerate(lens):
        own = order[at:at + need[i]]
        table[i, :need[i]] = own
        rows = torch.full((need[i] * page, 576), fill, dtype=dtype)
        rows[:l] = torch.randn(l, 576, generator=g).to(dtype)
        cache[own] = rows.view(-1, page, 576)
        at += need[i]
    return cache, table


def chunk_inputs(lens_q, lens, H, page, dtype, seed, **kw):
    g = torch.Generator().manual_seed(seed + 1)
    cache, table = paged(lens, page, dtype, seed, **kw)
    q = torch.randn(sum(lens_q), H, 192, generator=g).to(dtype)
    return q, cache, table, (torch.randn(H, 256, 512, generator=g) * 512 ** -0.5).to(dtype)


def run_chunk(q, cache, table, lens, w, lens_q, keys=None, **kw):
    keys = sum(l for l, n in zip(lens, lens_q) if n) if keys is None else keys
    return latent().latent_chunk(q.cuda(), cache.cuda(), table.cuda(), i32(lens), w.cuda(), cu(lens_q), keys, **kw)


CHUNKS = [
    # new tokens, cached rows, heads, page, type
    ([1], [1], 1, 16, BF),
    ([37], [237], 3, 64, BF),
    ([128], [128], 1, 64, FP),
    ([5, 129], [129, 300], 2, 16, FP),
    ([64, 65, 1], [127, 128, 300], 5, 32, BF),
    ([1, 0, 3, 130], [2, 500, 0, 256], 2, 64, BF),          # one without new tokens, one without rows
    ([300, 5], [100, 1], 2, 128, BF),                        # more new tokens than rows
    ([256, 1, 2], [257, 385, 1000], 17, 192, FP),            # pages of one and a half tiles
    ([7, 300], [9000, 310], 2, 64, BF),                      # keys shared by CTAs of the device's choice
    ([20], [4100], 2, 32, FP),                               # and of the host's
    ([700, 3], [2500, 2048], 2, 64, BF),                     # around the border of few keys: pairs of tiles on either side,
    ([300, 260, 2], [2049, 2049, 2050], 1, 16, BF),
    ([700, 200], [900, 257], 2, 64, FP),
    ([600] * 8 + [40], [900] * 8 + [2000], 6, 64, BF),       # two numbers a key with CTAs that share keys,
    ([2048], [2048], 1, 64, BF), ([40], [2040], 3, 32, BF),  # and in clusters
]


@pytest.mark.parametrize("lens_q,lens,H,page,dtype", CHUNKS)
def test_chunk(lens_q, lens, H, page, dtype):
    """NaN in the rows past each sequence's end and in unused pages, and in the workspace."""
    q, cache, table, w = chunk_inputs(lens_q, lens, H, page, dtype, seed=sum(lens), fill=float("nan"))
    keys = sum(l for l, n in zip(lens, lens_q) if n) + 5
    ws = torch.full((latent().latent_chunk_workspace_bytes(sum(lens_q), keys, H, len(lens)),), 255, dtype=torch.uint8, device="cuda")
    o, lse = run_chunk(q, cache, table, lens, w, lens_q, keys, workspace=ws)
    assert status(ws) == 0
    ro, rl, eo, el = sv.latent_chunk(q, cache, table, lens, w, lens_q, dtype=dtype, u=U[dtype], tiny=TINY[dtype], few=FEW[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")
    again = run_chunk(q, cache, table, lens, w, lens_q, keys)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("n,page,dtype", [(33, 16, BF), (70, 64, FP), (1100, 32, BF)])
def test_chunk_of_many_sequences(n, page, dtype):
    some = [0, 0, 1, 1, 2, 5, 31, 64]
    g = torch.Generator().manual_seed(n)
    lens_q = [some[i] for i in torch.randint(0, 8, (n,), generator=g).tolist()]
    lens = [l + e for l, e in zip(lens_q, torch.randint(0, 40 if n > 100 else 150, (n,), generator=g).tolist())]
    q, cache, table, w = chunk_inputs(lens_q, lens, 2, page, dtype, seed=n, fill=float("nan"))
    o, lse = run_chunk(q, cache, table, lens, w, lens_q)
    ro, rl, eo, el = sv.latent_chunk(q, cache, table, lens, w, lens_q, dtype=dtype, u=U[dtype], tiny=TINY[dtype], few=FEW[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


def test_chunk_scale_and_strided_inputs():
    lens_q, lens = [40, 9], [150, 60]
    q, cache, table, w = chunk_inputs(lens_q, lens, 2, 64, BF, seed=5, width=6)
    want = run_chunk(q, cache, table, lens, w, lens_q, scale=0.03)
    wide = torch.zeros(49, 4, 200, dtype=BF, device="cuda")
    wide[:, 1:3, 3:195] = q.cuda()
    tables = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    tables.copy_(table.T)
    big = torch.zeros(2, 256, 520, dtype=BF, device="cuda")
    big[..., 4:516] = w.cuda()
    got = latent().latent_chunk(wide[:, 1:3, 3:195], cache.cuda(), tables.T, i32(lens), big[..., 4:516], cu(lens_q), 210, scale=0.03)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ro, rl, eo, el = sv.latent_chunk(q, cache, table, lens, w, lens_q, scale=0.03, dtype=BF, u=U[BF], few=FEW[BF])
    near(want[0], ro, eo, "o")
    near(want[1], rl, el, "lse")


@pytest.mark.parametrize("page", [16, 64, 128])
def test_chunk_missing_pages_count_as_zeros(page):
    lens_q, lens = [10, 70, 3], [200, 300, 130]
    q, cache, table, w = chunk_inputs(lens_q, lens, 2, page, BF, seed=page, fill=float("nan"))
    table[0, 0], table[1, 1], table[2, -(-130 // page) - 1] = -1, cache.shape[0], 1 << 30
    ws = torch.zeros(latent().latent_chunk_workspace_bytes(83, 630, 2, 3), dtype=torch.uint8, device="cuda")
    o, lse = run_chunk(q, cache, table, lens, w, lens_q, workspace=ws)
    assert status(ws) == 8
    ro, rl, eo, el = sv.latent_chunk(q, cache, table, lens, w, lens_q, dtype=BF, u=U[BF], few=FEW[BF])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


def test_chunk_lengths_and_room_are_clipped_and_reported():
    lens_q, lens = [10, 20, 5], [100, 128, 60]
    q, cache, table, w = chunk_inputs(lens_q, lens, 2, 64, BF, seed=9)      # two columns: 128 rows at most
    ws = torch.zeros(latent().latent_chunk_workspace_bytes(35, 9300, 2, 3), dtype=torch.uint8, device="cuda")
    good = run_chunk(q, cache, table, lens, w, lens_q, workspace=ws)
    assert status(ws) == 0
    for keys in (288, 9300):                                                # 9300: with CTAs that share keys
        got = run_chunk(q, cache, table, [100, 1000, 60], w, lens_q, keys, workspace=ws)
        assert status(ws) == 8 and all(torch.equal(a, b) for a, b in zip(got, good))
        got = run_chunk(q, cache, table, [100, 128, -5], w, lens_q, keys, workspace=ws)
        assert status(ws) == 8 and torch.equal(got[0][:30], good[0][:30]) and (got[0][30:] == 0).all()
    got = run_chunk(q, cache, table, lens, w, lens_q, 228, workspace=ws)    # none left for the last one
    assert status(ws) == 8 and torch.equal(got[0][:30], good[0][:30])
    assert (got[0][30:] == 0).all() and torch.isinf(got[1][30:]).all()
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    run_chunk(q, cache, table, lens, w, lens_q, 0, workspace=small)
    assert status(small) == 8
    latent().latent_chunk(q.cuda(), cache.cuda(), table.cuda(), i32(lens), w.cuda(), i32([0, 10, 5, 35]), 288, workspace=ws)
    assert status(ws) == 4
    latent().latent_chunk(q.cuda(), cache.cuda(), table.cuda(), i32(lens), w.cuda(), i32([0, 10, 30, 36]), 288, workspace=ws)
    assert status(ws) == 4


def test_chunk_leaves_rows_behind_the_last_sequence():
    from chunked_gated_delta_kda_gb300 import binding
    lens_q, lens = [10, 20], [100, 128]
    q, cache, table, w = (t.cuda() for t in chunk_inputs(lens_q, lens, 2, 64, BF, seed=11))
    want = latent().latent_chunk(q, cache, table, i32(lens), w, cu(lens_q), 228)
    padded = torch.full((300, 2, 192), float("nan"), dtype=BF, device="cuda")
    padded[:30] = q
    o, lse = torch.full((300, 2, 128), 7.0, dtype=BF, device="cuda"), torch.full((300, 2), 7.0, device="cuda")
    lib = binding.load_library()
    for keys in (228, 9000):
        need = latent().latent_chunk_workspace_bytes(300, keys, 2, 2)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        n, c = i32(lens), cu(lens_q)
        rc = lib.kda_latent_chunk(padded.data_ptr(), cache.data_ptr(), cache.shape[0], 64, table.data_ptr(), table.shape[1],
                                  n.data_ptr(), w.data_ptr(), 0.0, c.data_ptr(), keys, o.data_ptr(), lse.data_ptr(), 300, 2, 2, 0,
                                  ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and status(ws) == 0
        assert torch.equal(o[:30], want[0]) and torch.equal(lse[:30], want[1]) and (o[30:] == 7).all() and (lse[30:] == 7).all()
    empty = latent().latent_chunk(q[:0], cache, table, i32(lens), w, i32([0, 0, 0]), 0)
    assert empty[0].shape == (0, 2, 128)


def test_chunk_captured_and_replayed_with_other_lengths():
    lens_q, lens = [10, 20], [100, 128]
    q, cache, table, w = (t.cuda() for t in chunk_inputs(lens_q, lens, 2, 64, BF, seed=12))
    n, c = i32([128, 128]), i32([0, 15, 30])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        latent().latent_chunk(q, cache, table, n, w, c, 256)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = latent().latent_chunk(q, cache, table, n, w, c, 256)
    for lq, lk in (([15, 15], [128, 128]), (lens_q, lens), ([30, 0], [31, 5])):
        n.copy_(i32(lk))
        c.copy_(cu(lq))
        graph.replay()
        want = latent().latent_chunk(q, cache, table, i32(lk), w, cu(lq), 256)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_chunk_past_32_bit_offsets():
    """Expanded rows of more than 2^31 elements: the last sequence gets the bits that it gets alone."""
    H, page, lens = 128, 64, [8200] * 8 + [300]
    assert sum(lens) * H * 256 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(13)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    need = -(-8200 // page)
    cache, w, q = r(8 * need + 5, page, 576), r(H, 256, 512) * 512 ** -0.5, r(8 + 20, H, 192)
    table = torch.zeros(9, need, dtype=torch.int32, device="cuda")
    table[:8] = torch.arange(8 * need, device="cuda").view(8, need)
    table[8, :5] = torch.arange(8 * need, 8 * need + 5, device="cuda")
    o, lse = latent().latent_chunk(q, cache, table, i32(lens), w, cu([1] * 8 + [20]), sum(lens))
    a, b = latent().latent_chunk(q[8:], cache, table[8:], i32(lens[8:]), w, cu([20]), 300)
    assert torch.equal(o[8:], a) and torch.equal(lse[8:], b)


def test_chunk_waits_that_run_out_are_reported():
    from chunked_gated_delta_kda_gb300 import binding
    lens_q, lens = [100, 20], [600, 128]
    q, cache, table, w = (t.cuda() for t in chunk_inputs(lens_q, lens, 3, 64, BF, seed=14))
    ws = torch.zeros(latent().latent_chunk_workspace_bytes(120, 728, 3, 2), dtype=torch.uint8, device="cuda")
    args = q, cache, table, i32(lens), w, cu(lens_q), 728
    want = latent().latent_chunk(*args, workspace=ws)
    binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 1)
    try:
        latent().latent_chunk(*args, workspace=ws)
        assert status(ws) == 5
    finally:
        binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 0)
    got = latent().latent_chunk(*args, workspace=ws)
    assert status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# drafts
def draft_inputs(N, S, V, dtype, seed, none=False, ragged=False):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(N, S + 1, V, generator=g) * 2
    target = torch.softmax(logits, -1).to(dtype)
    draft = torch.softmax(logits[:, :S] + torch.randn(N, S, V, generator=g), -1).to(dtype)
    if S:
        tokens = torch.multinomial(draft.float().reshape(-1, V), 1, generator=g).reshape(N, S)
    else:
        tokens = torch.zeros(N, 0, dtype=torch.int64)
    if ragged:
        tokens = torch.where(torch.arange(S) < torch.randint(0, S + 1, (N, 1), generator=g), tokens, -1)
    return tokens, target, torch.rand(N, S + 1, generator=g), None if none else draft


def check_drafts(tokens, target, uniform, draft, got=None, slack=2.0 ** -44):
    if got is None:
        got = verify(tokens.cuda(), target.cuda(), uniform.cuda(), None if draft is None else draft.cuda())
    out, accepted = got[0].cpu(), got[1].cpu()
    S = tokens.shape[1]
    for n, (a, allowed) in enumerate(sv.verify_drafts(tokens, target, uniform, draft, slack=slack)):
        assert accepted[n] == a + 1 and out[n, :a].tolist() == tokens[n, :a].tolist(), (n, a)
        assert (out[n, a + 1:] == -1).all() and out.shape == (len(out), S + 1)
        if allowed is None:
            assert 0 <= out[n, a] < target.shape[2]
        else:
            assert out[n, a] in allowed, (n, a, out[n, a], allowed)


@pytest.mark.parametrize("N,S,V,dtype", [
    (1, 4, 32768, F32), (3, 5, 50257, BF), (2, 1, 70001, F32), (40, 3, 1, F32), (40, 3, 2, BF), (30, 33, 100, FP),
    (9, 0, 513, F32), (5, 70, 511, BF), (7, 2, 8192, FP), (7, 2, 8193, F32), (3, 2, 65537, F32), (300, 2, 40, F32)])
@pytest.mark.parametrize("none", [False, True])
def test_drafts(N, S, V, dtype, none):
    check_drafts(*draft_inputs(N, S, V, dtype, seed=N * V + S, none=none, ragged=V % 2 == 1))


def test_drafts_in_slices_of_a_padded_vocabulary():
    tokens, target, u, draft = draft_inputs(4, 3, 1000, F32, seed=2)
    for width, first in ((1024, 0), (1001, 1), (1027, 3)):
        wide = torch.full((4, 5, width), float("nan"), device="cuda")
        wide[:, :4, first:first + 1000] = target.cuda()
        other = torch.full((4, 3, width + 4), float("nan"), device="cuda")
        other[..., :1000] = draft.cuda()
        check_drafts(tokens, target, u, draft, verify(tokens.cuda(), wide[:, :4, first:first + 1000], u.cuda(), other[..., :1000]))
    turned = target.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    check_drafts(tokens, target, u, draft, verify(tokens.cuda(), turned, u.cuda(), draft.cuda()))


@pytest.mark.parametrize("V", [16, 1024, 4096, 65536])
def test_drafts_at_borders(V):
    """Probabilities of whole parts of V and uniform numbers on the borders: the sums are exact, and the border's own
    token is not the one below it; the largest number below 1 draws the last token with weight."""
    k = torch.randint(0, V, (50,), generator=torch.Generator().manual_seed(V))
    target = torch.full((50, 1, V), 1.0 / V)
    out, n = verify(torch.zeros(50, 0, dtype=torch.int64, device="cuda"), target.cuda(), (k / V)[:, None].cuda())
    assert torch.equal(out[:, 0].cpu(), k) and (n == 1).all()
    target[:, :, V // 2:] = 0
    last = torch.full((50, 1), 1 - 2.0 ** -24)
    out, _ = verify(torch.zeros(50, 0, dtype=torch.int64, device="cuda"), target.cuda(), last.cuda())
    assert (out == V // 2 - 1).all()
    out, _ = verify(torch.zeros(50, 0, dtype=torch.int64, device="cuda"), target.cuda(), torch.ones(50, 1, device="cuda"))
    assert (out == V // 2 - 1).all()                     # (1 itself is past the border of every token)


def test_drafts_small_numbers_beside_large_ones():
    """Weights from 1 to 2^-140, where a 32-bit sum would lose them all; the border stands among the small ones."""
    V = 3000
    target = torch.full((20, 1, V), 2.0 ** -30)
    target[:, 0, 0] = 1.0
    target[:, 0, 1::7] = 2.0 ** -140
    u = torch.full((20, 1), 1 - 2.0 ** -24)
    check_drafts(torch.zeros(20, 0, dtype=torch.int64), target, u, None)
    target[:, 0, 0], target[:, 0, -1] = 2.0 ** -30, 1.0
    u = (torch.arange(20) * 2.0 ** -27)[:, None]
    check_drafts(torch.zeros(20, 0, dtype=torch.int64), target, u, None)
    p = torch.rand(20, 2, V, generator=torch.Generator().manual_seed(1)) * 2.0 ** -12
    q = p[:, :1] * (1 + 2.0 ** -23 * torch.randint(-2, 3, (20, 1, V), generator=torch.Generator().manual_seed(2)))
    check_drafts(torch.zeros(20, 1, dtype=torch.int64), p, torch.full((20, 2), 1 - 2.0 ** -20), q)   # p - q of a few last bits


def test_drafts_that_are_equal_or_odd_numbers():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    p = torch.softmax(torch.randn(6, 3, 700, generator=torch.Generator().manual_seed(3)), -1)
    d = torch.zeros(6, 2, dtype=torch.int64)
    u = torch.full((6, 3), 0.4)
    u[3:, 0] = 1.0                                       # not below p / q = 1, and p - q has no weight: p itself
    check_drafts(d, p, u, p[:, :2].clone(), verify(d.cuda(), p.cuda(), u.cuda(), p[:, :2].cuda(), workspace=ws))
    assert status(ws) == 0
    x = p.clone()
    x[:, :, ::3], x[:, :, 1::9] = float("nan"), -1.0     # no weight
    check_drafts(d, x, u, p[:, :2].clone(), verify(d.cuda(), x.cuda(), u.cuda(), p[:, :2].cuda(), workspace=ws))
    assert status(ws) == 0
    for bad in (x * 0, torch.full_like(p, float("nan")), torch.full_like(p, float("inf"))):
        out, n = verify(torch.full((6, 2), -1, device="cuda"), bad.cuda(), u.cuda(), workspace=ws)
        assert status(ws) == 9 and (n == 1).all() and ((out[:, 0] >= 0) & (out[:, 0] < 700)).all() and (out[:, 1:] == -1).all()
    d[2, 1] = 700                                        # past the vocabulary: the drafts end before it
    u[2] = 0.0
    out, n = verify(d.cuda(), p.cuda(), u.cuda(), p[:, :2].cuda(), workspace=ws)
    assert status(ws) == 9 and n[2] == 2
    check_drafts(d, p, u, p[:, :2].clone(), (out, n))
    verify(d[:2].cuda(), p[:2].cuda(), u[:2].cuda(), p[:2, :2].cuda(), workspace=ws)
    assert status(ws) == 0


def test_drafts_past_32_bit_offsets():
    V, N = 140000, 4000                                  # 2 rows of 140000 a sequence: 2.2 GB of bf16, 1.1e9 elements each
    target = torch.zeros(N, 4, V, dtype=BF, device="cuda")
    assert target.numel() > 2 ** 31
    at = torch.arange(N, device="cuda") % V
    target[torch.arange(N, device="cuda"), 2, at * 31 % V] = 1.0
    target[:, :2, 5] = 1.0
    out, n = verify(torch.tensor([[5, 5, -1]], device="cuda").expand(N, 3), target, torch.full((N, 4), 0.5, device="cuda"))
    assert (n == 3).all() and torch.equal(out[:, 2], at * 31 % V) and (out[:, :2] == 5).all() and (out[:, 3] == -1).all()


# ---------------------------------------------------------------------------
# pages
def pool_state(lens, page, spare, seed, group=1, width=None):
    """Tables of requests whose first pages are the group's first one's: (table, refs, free list, head)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-l // page) for l in lens]
    shared = [0 if i % group == 0 else min(need[i], need[i - i % group]) // 2 for i in range(len(lens))]
    used = sum(need) - sum(shared)
    order = torch.randperm(used + spare, generator=g).tolist()
    width = width or max(1, max(need))
    table = torch.randint(-3, used + spare + 3, (len(lens), width), generator=g).to(torch.int32)   # anything behind
    refs, at = [0] * (used + spare), 0
    for i, n in enumerate(need):
        lead = i - i % group
        row = table[lead, :shared[i]].tolist() + order[at:at + n - shared[i]]
        table[i, :n] = torch.tensor(row, dtype=torch.int32)
        for p in row[:shared[i]]:
            refs[p] += 1
        at += n - shared[i]
    return table, refs, order, used


STATES = [
    # requests' longest length, how many, page, spare pages, group
    (1, 1, 1, 1, 1), (100, 7, 16, 5, 2), (300, 40, 24, 400, 4), (4000, 64, 16, 9000, 3), (70, 3000, 64, 10, 2),
    (20000, 100, 7, 30000, 2),
]


def lengths(n, longest, seed):
    g = torch.Generator().manual_seed(seed)
    return [0 if x % 5 == 3 else x % (longest + 1) for x in torch.randint(0, 1 << 30, (n,), generator=g).tolist()]


@pytest.mark.parametrize("longest,n,page,spare,group", STATES)
def test_page_free(longest, n, page, spare, group):
    lens = lengths(n, longest, n)
    table, refs, free, head = pool_state(lens, page, spare, n, group)
    keep = [0 if i % 3 == 0 else l if i % 3 == 1 else l * (i % 7) // 7 for i, l in enumerate(lens)]
    t, f = table.cuda(), i32(free)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):                                   # the inputs but for the listed pages stay as they are
        got = pages().page_free(t, i32(lens), i32(keep), i32(refs), f, i32([head]), page, workspace=ws)
        wl, wr, wf, wh = sv.page_free(table, lens, keep, refs, free, head, page)
        shared = any(k < l and k % page and wr[table[i, k // page]] > 0 for i, (k, l) in enumerate(zip(keep, lens)))
        assert status(ws) == (8 if shared else 0) and torch.equal(t.cpu(), table)
        assert got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh and f.tolist() == wf


@pytest.mark.parametrize("longest,n,page,spare,group", STATES)
def test_page_fork(longest, n, page, spare, group):
    lens = lengths(n, longest, n + 1)
    table, refs, free, head = pool_state(lens, page, spare, n, group)
    empty = [i for i in range(n) if lens[i] == 0]
    children = empty + [-1, -5]
    g = torch.Generator().manual_seed(n)
    order = torch.randperm(len(children), generator=g).tolist()
    children = [children[i] for i in order]
    parents = torch.randint(0, n, (len(children),), generator=g).tolist()
    room = len(free) - head
    for i, a in enumerate(parents):                      # no more own pages than there are
        if children[i] >= 0 and lens[a] % page:
            room -= 1
            if room < 0:
                children[i] = -1
    t = table.cuda()
    for _ in range(2):
        got = pages().page_fork(t, i32(lens), i32(parents), i32(children), i32(refs), i32(free), i32([head]), page)
        wt, wl, wr, wh, wp = sv.page_fork(table, lens, parents, children, refs, free, head, page)
        assert torch.equal(t.cpu(), wt)
        assert got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh
        assert [tuple(p) for p in got[3].tolist()] == wp
    some = [lens[a] * (i % 5) // 4 for i, a in enumerate(parents)]
    for i, (a, c) in enumerate(zip(parents, children)):
        if some[i] % page and not lens[a] % page and c >= 0:   # (there are own pages for parents whose last page is not full)
            some[i] -= some[i] % page
    t = table.cuda()
    got = pages().page_fork(t, i32(lens), i32(parents), i32(children), i32(refs), i32(free), i32([head]), page, fork_lens=i32(some))
    wt, wl, wr, wh, wp = sv.page_fork(table, lens, parents, children, refs, free, head, page, some)
    assert torch.equal(t.cpu(), wt) and got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh
    assert [tuple(p) for p in got[3].tolist()] == wp


@pytest.mark.parametrize("longest,n,page,spare,group", STATES)
def test_page_compact(longest, n, page, spare, group):
    lens = lengths(n, longest, n + 2)
    table, refs, free, head = pool_state(lens, page, spare, n, group)
    got = pages().page_compact(table.cuda(), i32(lens), i32(refs), i32(free), i32([head]), page)
    wt, wr, wf, wp, wc, wm = sv.page_compact(table, lens, refs, free, head, page)
    assert torch.equal(got[0].cpu(), wt) and got[1].tolist() == wr and got[2].tolist() == wf
    assert [tuple(p) for p in got[3].tolist()] == wp and got[4].item() == wc and got[5].tolist() == wm


@pytest.mark.parametrize("P", [1, 2, 7, 9, 255, 256, 257, 4096, 32769, 300001, 2 ** 20, 2 ** 20 + 1])
def test_pages_of_any_number(P):
    """One request on every second page; all of it freed again; none in use, and all."""
    for held in {0, P // 2, P}:
        order = torch.cat([torch.arange(0, P, 2), torch.arange(1, P, 2)]).flip(0)
        table = order[:held][None].to(torch.int32)
        table = table if held else torch.zeros(1, 1, dtype=torch.int32)
        refs = torch.zeros(P, dtype=torch.int32)
        f, lens = order.to(torch.int32), [held]
        got = pages().page_free(table.cuda(), i32(lens), i32([0]), refs.cuda(), f.cuda(), i32([held]), 1)
        assert got[2].item() == 0 and not got[1].any()
        mine = f.cuda()
        pages().page_free(table.cuda(), i32(lens), i32([0]), refs.cuda(), mine, i32([held]), 1)
        assert torch.equal(mine[:held].cpu(), f[:held].sort().values) and torch.equal(mine[held:].cpu(), f[held:])
        t, r, free, pairs, count, moved = (x.cpu() for x in pages().page_compact(
            table.cuda(), i32(lens), refs.cuda(), f.cuda(), i32([held]), 1))
        assert torch.equal(free, torch.cat([f[:held], torch.arange(held, P, dtype=torch.int32)]))
        if held:
            assert torch.equal(t[0].sort().values, torch.arange(held, dtype=torch.int32)) and torch.equal(moved[table[0].long()], t[0])
        k = count.item()
        assert (pairs[k:] == -1).all() and (pairs[:k, 0] >= held).all() and (pairs[:k, 1] < held).all()
        assert torch.equal(moved[pairs[:k, 0].long()], pairs[:k, 1]) and (pairs[:k].diff(dim=0) > 0).all()


def test_page_faults_are_reported():
    """A page outside the pool, one that loses more owners than it has, lengths out of range, rows that are no rows, a
    child twice or with tokens, a free list that ends: what is right beside them stays right."""
    p = pages()
    table = torch.tensor([[4, 5, 6], [4, 9, -1], [-1, -1, -1], [-1, -1, -1], [2, 2, 2]], dtype=torch.int32)
    lens, refs, free = [10, 8, 0, 0, 8], [0, 0, 0, 0, 1, 0, 0, 0], [4, 5, 6, 2, 3, 0, 1, 7]
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")

    def fork(parents, children, lens=lens, free=free, head=4, page=4):
        t = table.cuda()
        got = p.page_fork(t, i32(lens), i32(parents), i32(children), i32(refs), i32(free), i32([head]), page, workspace=ws)
        return status(ws), t.tolist(), *(x.tolist() for x in got)

    s, t, l, r, h, pairs = fork([0, 0], [2, 3])
    assert s == 0 and t[2] == [4, 5, 3] and t[3] == [4, 5, 0] and r == [0, 0, 0, 0, 3, 2, 0, 0] and h == [6] and pairs == [[6, 3], [6, 0]]
    for parents, children in (([0, 0], [2, 2]), ([0, 7], [2, 3]), ([0, -1], [2, 3]), ([0, 0], [2, 9]), ([0, 0], [2, 1])):
        s, t, l, r, h, pairs = fork(parents, children)
        assert s == 8 and t[2] == [4, 5, 3] and t[3] == [-1] * 3 and l == [10, 8, 10, 0, 8] and h == [5] and pairs == [[6, 3], [-1, -1]]
    s, t, l, r, h, pairs = fork([1], [3])                 # its second page does not exist
    assert s == 8 and t[3] == [4, -1, -1] and l[3] == 8 and r[4] == 2 and pairs == [[-1, -1]]
    s, t, l, r, h, pairs = fork([0, 0], [2, 3], head=7)   # one page left
    assert s == 8 and t[2] == [4, 5, 7] and t[3] == [4, 5, -1] and h == [8] and pairs == [[6, 7], [-1, -1]]
    for some, kept in ((11, 10), (-1, 0)):                # tokens that the parent has not
        t = table.cuda()
        got = p.page_fork(t, i32(lens), i32([0]), i32([2]), i32(refs), i32(free), i32([4]), 4, fork_lens=i32([some]), workspace=ws)
        assert status(ws) == 8 and got[0].tolist()[2] == kept
    for n in (99, -4):
        s, t, l, r, h, pairs = fork([0, 4], [2, 3], lens=[10, 8, 0, 0, n])
        assert s == 8 and t[2] == [4, 5, 3] and l[2] == 10 and l[3] == (12 if n > 0 else 0)

    def release(keep, lens=lens, head=4, refs=refs):
        f = i32(free)
        got = p.page_free(table.cuda(), i32(lens), i32(keep), i32(refs), f, i32([head]), 4, workspace=ws)
        return status(ws), f.tolist(), *(x.tolist() for x in got)

    s, f, l, r, h = release([4, 4, 0, 0, 8])
    assert s == 8                                         # page 9
    s, f, l, r, h = release([4, 8, 0, 0, 8])
    assert s == 0 and f == [4, 5, 5, 6, 3, 0, 1, 7] and h == [2] and l == [4, 8, 0, 0, 8]
    s, f, l, r, h = release([10, 8, 0, 0, 0])             # page 2 twice
    assert s == 8 and h == [3] and f[3] == 2 and r == refs
    s, f, l, r, h = release([3, 5, 0, 0, 8])              # into page 4, which the other one owns too
    assert s == 8 and l == [3, 5, 0, 0, 8] and r == [0, 0, 0, 0, 1, 0, 0, 0] and h == [2]
    s, f, l, r, h = release([3, 0, 0, 0, 8], lens=[10, 4, 0, 0, 8])   # which ends
    assert s == 0 and l == [3, 0, 0, 0, 8] and r == [0] * 8 and h == [2]
    s, f, l, r, h = release([11, -1, 0, 0, 8])
    assert s == 8 and l == [10, 0, 0, 0, 8] and r[4] == 0 and h == [4]
    s, f, l, r, h = release([0, 8, 0, 0, 8], head=1)      # no room in front
    assert s == 8 and h == [0] and f == [6, 5, 6, 2, 3, 0, 1, 7]
    s, f, l, r, h = release([0, 8, 0, 0, 8], lens=[1000, 8, 0, 0, 8])
    assert s == 0 or s == 8

    def compact(table=table, lens=[10, 4, 0, 0, 4], free=free, head=4):
        got = p.page_compact(table.cuda(), i32(lens), i32(refs), i32(free), i32([head]), 4, workspace=ws)
        return status(ws), *(x.tolist() for x in got)

    s, t, r, f, pairs, count, moved = compact()
    assert s == 0 and pairs == [[4, 0], [5, 1], [6, 3], [-1, -1]] and count == [3] and moved == [-1, -1, 2, -1, 0, 1, 3, -1]
    assert t == [[0, 1, 3], [0, -1, -1], [-1] * 3, [-1] * 3, [2, -1, -1]] and r == [1] + [0] * 7 and f == [4, 5, 6, 2, 4, 5, 6, 7]
    assert compact(free=[4, 5, 6, 2, 3, 0, 1, 1])[0] == 8 and compact(free=[4, 5, 6, 2, 3, 0, 1, 8])[0] == 8
    assert compact(lens=[10, 8, 0, 0, 4])[0] == 8 and compact(lens=[10, 4, 99, 0, 4])[0] == 8 and compact(lens=[10, 4, -1, 0, 4])[0] == 8
    assert compact(head=3)[0] == 8                        # page 2 is held and free
    assert compact(table=table[:, :0], lens=[0] * 5)[0] == 0


@pytest.mark.parametrize("F", [255, 256, 257, 1024, 1025, 2500])
def test_many_forks_with_children_twice(F):
    """Every third entry wants a child that an earlier one has, some far before it."""
    rows = F + 5
    lens = [33, 16] + [0] * (rows - 2)
    table = torch.full((rows, 4), -1, dtype=torch.int32)
    table[0, :3], table[1, 0] = torch.tensor([0, 1, 2]), 3
    refs, free = [0] * (F + 10), list(range(F + 10))
    order = torch.randperm(rows - 2, generator=torch.Generator().manual_seed(F)).tolist()
    children = [order[i] + 2 if i % 3 or i < 9 else order[i // 3 if i % 2 else i - 1] + 2 for i in range(F)]
    parents = [i % 2 for i in range(F)]
    twice = [c in children[:i] for i, c in enumerate(children)]
    assert sum(twice) > F // 4
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    t = table.cuda()
    got = pages().page_fork(t, i32(lens), i32(parents), i32(children), i32(refs), i32(free), i32([4]), 16, workspace=ws)
    wt, wl, wr, wh, wp = sv.page_fork(table, lens, parents, [-1 if d else c for c, d in zip(children, twice)], refs, free, 4, 16)
    assert status(ws) == 8 and torch.equal(t.cpu(), wt) and got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh
    assert [tuple(p) for p in got[3].tolist()] == wp


def test_page_tensors_that_start_anywhere():
    """Views whose first element is not on 16 bytes, and a table that is a slice."""
    lens = lengths(30, 200, 3)
    table, refs, free, head = pool_state(lens, 16, 50, 3, 2)
    shift = lambda x: torch.cat([torch.zeros(3, dtype=torch.int32, device="cuda"), i32(x)])[3:]  # noqa: E731
    wide = torch.zeros(30, table.shape[1] + 5, dtype=torch.int32, device="cuda")
    wide[:, 2:-3] = table.cuda()
    keep = [l // 2 for l in lens]
    f = shift(free)
    got = pages().page_free(wide[:, 2:-3], shift(lens), shift(keep), shift(refs), f, shift([head]), 16)
    wl, wr, wf, wh = sv.page_free(table, lens, keep, refs, free, head, 16)
    assert got[0].tolist() == wl and got[1].tolist() == wr and got[2].item() == wh and f.tolist() == wf
    got = pages().page_compact(wide[:, 2:-3], shift(lens), shift(refs), shift(free), shift([head]), 16)
    wt, wr, wf, wp, wc, wm = sv.page_compact(table, lens, refs, free, head, 16)
    assert torch.equal(got[0].cpu(), wt) and got[1].tolist() == wr and got[2].tolist() == wf and got[5].tolist() == wm
    child = lens.index(0)
    a = max(range(30), key=lambda i: lens[i])
    t = table.cuda()
    got = pages().page_fork(t, shift(lens), shift([a]), shift([child]), shift(refs), shift(free), shift([head]), 16)
    wt, wl, wr, wh, wp = sv.page_fork(table, lens, [a], [child], refs, free, head, 16)
    assert torch.equal(t.cpu(), wt) and got[0].tolist() == wl and got[1].tolist() == wr
    with pytest.raises(ValueError, match="contiguous"):
        pages().page_fork(wide[:, 2:-3], shift(lens), shift([a]), shift([child]), shift(refs), shift(free), shift([head]), 16)
    with pytest.raises(ValueError, match="contiguous"):
        pages().page_free(t, i32(lens), i32(keep), i32(refs), i32(free + free)[::2], i32([head]), 16)


@pytest.mark.parametrize("shape,dtype,pools", [((9, 64, 576), BF, 3), ((300, 4), F32, 1), ((7, 2, 128, 128), F32, 2),
                                               ((50, 3, 24), FP, 70), ((33, 16, 576), FP, 65)])
def test_page_copy(shape, dtype, pools):
    g = torch.Generator().manual_seed(shape[0])
    before = [torch.randn(shape, generator=g).to(dtype) for _ in range(pools)]
    order = torch.randperm(shape[0], generator=g).tolist()
    half = shape[0] // 2
    pairs = [(order[i % half], order[half + i]) for i in range(shape[0] - half)]
    pairs.insert(1, (-1, -1))
    pairs.insert(3, (order[0], -1))
    at = [t.cuda() for t in before]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    for count, upto in ((None, len(pairs)), (i32([3]), 3), (i32([0]), 0), (i32([1000]), len(pairs)), (i32([-3]), 0)):
        for t, b in zip(at, before):
            t.copy_(b)
        got = pages().page_copy(at if pools > 1 else at[0], i32(pairs), count=count, workspace=ws)
        assert status(ws) == 0
        for t, b in zip(got if pools > 1 else [got], before):
            want = b.clone()
            for s, d in pairs[:upto]:
                if s >= 0 and d >= 0:
                    want[d] = b[s]
            assert torch.equal(t.cpu(), want)
    pages().page_copy(at, i32([(0, shape[0])]), workspace=ws)
    assert status(ws) == 8
    pages().page_copy(at, i32([]).view(0, 2), workspace=ws)
    assert status(ws) == 0


def test_page_copy_refusals_and_large_pools():
    p = pages()
    x = torch.zeros(4, 6, dtype=F32, device="cuda")
    for pools, match in ((x, "16 bytes"), (torch.zeros(33, device="cuda")[1:].view(4, 8), "16 bytes"), (torch.zeros(4, 16, device="cuda")[:, :8], "contiguous"),
                         ([torch.zeros(4, 8, device="cuda"), torch.zeros(5, 8, device="cuda")], "one shape"), (x[:0], "16 bytes")):
        with pytest.raises(ValueError, match=match):
            p.page_copy(pools, i32([(0, 1)]))
    big = torch.zeros(140000, 16 * 576, dtype=BF, device="cuda")      # 2.6 GB, pages past 2^31 bytes
    big[3] = 1.0
    p.page_copy(big, i32([(3, 139999), (139998, 3)]))
    assert (big[139999] == 1).all() and (big[3] == 0).all()


def test_calls_are_captured_and_run_on_other_streams():
    lens = lengths(20, 300, 5)
    table, refs, free, head = pool_state(lens, 16, 40, 5, 2)
    keep = [l // 2 for l in lens]
    t, n, k, r, f, h = table.cuda(), i32(lens), i32(keep), i32(refs), i32(free), i32([head])
    tokens, target, u, draft = (x.cuda() for x in draft_inputs(3, 2, 3000, F32, seed=8))
    pool = torch.randn(len(refs), 64, device="cuda")

    def work():
        a = verify(tokens, target, u, draft)
        b = pages().page_free(t, n, k, r, f, h, 16)
        c = pages().page_compact(t, n, r, f, h, 16)
        pages().page_copy(pool, c[3], count=c[4])
        return *a, *b, *c, pool.clone()

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for x in captured:
        x.zero_()
    graph.replay()
    for a, b, c in zip(want, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_wrappers_name_what_they_refuse():
    """On CUDA tensors, where each check can be reached."""
    z = lambda *s, d=torch.int32: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    with pytest.raises(TypeError, match="w_up"):
        latent().latent_chunk(z(4, 2, 192, d=BF), z(3, 16, 576, d=BF), z(1, 2), z(1), z(2, 256, 512, d=FP), z(2), 4)
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        latent().latent_chunk(z(4, 2, 192, d=BF), z(3, 16, 576, d=BF), z(1, 2), z(1), z(2, 256, 512, d=BF), z(1), 4)
    with pytest.raises(ValueError, match="num_keys"):
        latent().latent_chunk(z(4, 2, 192, d=BF), z(3, 16, 576, d=BF), z(1, 2), z(1), z(2, 256, 512, d=BF), z(2), 2 ** 33)
    with pytest.raises(ValueError, match="keep_lens"):
        pages().page_free(z(2, 3), z(2), z(3), z(4), z(4), z(1), 16)
    with pytest.raises(ValueError, match="parents"):
        pages().page_fork(z(2, 3), z(2), z(2), z(1), z(4), z(4), z(1), 16)
    with pytest.raises(ValueError, match="free_pages"):
        pages().page_compact(z(2, 3), z(2), z(4), torch.zeros(4, dtype=torch.int32), z(1), 16)
    with pytest.raises(TypeError, match="target_probs"):
        verify(z(1, 1, d=torch.int64), z(1, 2, 4, d=torch.float64), z(1, 2, d=F32))
    with pytest.raises(ValueError, match="uniform"):
        verify(z(1, 1, d=torch.int64), z(1, 2, 4, d=F32), z(1, 1, d=F32))


# ---------------------------------------------------------------------------
# together
def layers(n, requests, pages=64, **kw):
    from chunked_gated_delta_kda_gb300.latent_serving import LatentLayer
    return [LatentLayer(128, 2, requests, pages=pages, width=16, page_size=16, **kw) for _ in range(n)]


def test_layer_reads_a_prompt_in_chunks_forks_it_and_takes_tokens_back():
    """Whatever the steps, pages and forks were, a request's rows are those of a layer that read its tokens at once."""
    g = torch.Generator(device="cuda").manual_seed(5)
    layer, = layers(1, 4)
    x = torch.randn(4, 200, 128, generator=g, device="cuda").to(BF)
    tokens = [x[0, :0]] * 4

    def add(*counts):
        new = [x[i, len(tokens[i]):len(tokens[i]) + n] for i, n in enumerate(counts)]
        out = layer.chunk(torch.cat(new), i32(counts))
        for i, n in enumerate(new):
            tokens[i] = torch.cat([tokens[i], n])
        return out, counts

    def keep(*lens):
        layer.keep(i32(lens))
        for i, n in enumerate(lens):
            tokens[i] = tokens[i][:n]

    def check(out, counts):
        fresh, = layers(1, 4)
        want = fresh.prefill(torch.cat(tokens), i32([len(t) for t in tokens]))
        at = 0
        for i, n in enumerate(counts):
            end = sum(len(t) for t in tokens[:i + 1])
            a, b = out[at:at + n].float(), want[end - n:end].float()
            # as many rows in another product: a rounding of rows, queries, keys, values and output each, and the weights'
            assert (a - b).norm() <= 6 * 2.0 ** -8 * b.norm(), (i, n)
            at += n
        # every page has as many owners as the tables say, and the free list has the others
        held = [layer.table[i, :-(-len(t) // 16)].tolist() for i, t in enumerate(tokens)]
        owners = [sum(p in h for h in held) for p in range(64)]
        free = layer.free[layer.head.item():].tolist()
        assert layer.refs.tolist() == [max(o - 1, 0) for o in owners]
        assert sorted(free) == [p for p in range(64) if owners[p] == 0] and layer.lens.tolist() == [len(t) for t in tokens]

    check(*add(50, 20, 0, 0))
    check(*add(40, 1, 0, 0))
    layer.fork(i32([0, 0]), i32([2, 3]))
    tokens[2] = tokens[3] = tokens[0]
    x[2, :90] = x[3, :90] = x[0, :90]
    check(*add(7, 0, 7, 33))                               # into each one's own last page
    keep(97, 0, 92, 80)                                    # request 1 ends, 3 goes back into shared pages' tokens
    check(*add(3, 60, 5, 0))
    keep(0, 60, 97, 80)
    moved = layer.compact()
    assert moved > 0 and max(layer.table[i, :-(-n // 16)].max().item() for i, n in enumerate([0, 60, 97, 80]) if n) < 64 - len(
        layer.free[layer.head.item():])
    check(*add(10, 0, 1, 0))                               # into a page of a forked request: its own


def test_layer_does_not_go_back_into_a_shared_page():
    """A request that goes back into a page that others own too would write into their rows: refused; a fork of its first
    tokens has a page of its own."""
    layer, = layers(1, 2)
    x = torch.randn(60, 128, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(BF)
    layer.chunk(x[:48], i32([48, 0]))
    layer.fork(i32([0]), i32([1]))
    from chunked_gated_delta_kda_gb300 import binding
    with pytest.raises(binding.KdaError) as e:
        layer.keep(i32([48, 40]))
    assert e.value.code == 8
    assert layer.lens.tolist() == [48, 48]
    layer.keep(i32([48, 0]))
    layer.fork(i32([0]), i32([1]), i32([40]))
    assert layer.lens.tolist() == [48, 40] and layer.table[0, 2] != layer.table[1, 2]
    rows = lambda i: layer.cache[layer.table[i, :3].long()].reshape(-1, 576)  # noqa: E731
    assert torch.equal(rows(0)[:40], rows(1)[:40])
    layer.chunk(x[48:60], i32([0, 12]))
    layer.keep(i32([48, 32]))
    layer.keep(i32([0, 32]))                               # the other owner ends
    layer.keep(i32([0, 20]))


def test_drafts_leave_greedy_decoding_as_it_is():
    """Tokens of the largest probability, with drafts of every quality: the tokens are those without drafts."""
    from chunked_gated_delta_kda_gb300.latent_serving import Decoder
    g = torch.Generator(device="cuda").manual_seed(7)
    prompt = torch.randint(0, 50, (70,), generator=g, device="cuda")
    plain, quick = (Decoder(50, 256, 4, 2, pages=64, width=16, page_size=16, temper=1e4, seed=2) for _ in range(2))
    n = i32([40, 30])
    u = lambda s: torch.rand(2, s, generator=g, device="cuda")  # noqa: E731
    first = plain.start(prompt, n, u(1)[:, 0])
    assert torch.equal(first, quick.start(prompt, n, u(1)[:, 0]))
    want = [first]
    for _ in range(24):
        want.append(plain.step(want[-1], first.new_empty(2, 0), u(1))[0][:, 0])
    want = torch.stack(want, 1)
    texts, steps = [[t] for t in first.tolist()], 0
    while min(len(t) for t in texts) < 25:
        guess = torch.full((2, 3), -1, dtype=torch.int64, device="cuda")
        for i, t in enumerate(texts):
            right = (want[i].tolist() + [0] * 99)[len(t):len(t) + 3]
            wrong = [(r + 1) % 50 for r in right]
            kind = (steps + i) % 4                          # none; wrong from the first, the second, none of them on
            guess[i] = torch.tensor([[-1] * 3, wrong, right[:1] + wrong[1:], right][kind], device="cuda")
        out, count = quick.step(torch.tensor([t[-1] for t in texts], device="cuda"), guess, u(4))
        for t, row, c in zip(texts, out.tolist(), count.tolist()):
            t += row[:c]
        steps += 1
    for i in range(2):
        assert texts[i][:25] == want[i].tolist()
    assert steps < 24


def test_serving_example_runs():
    from chunked_gated_delta_kda_gb300 import latent_serving
    assert latent_serving.continue_forked() >= 1.0


def test_verified_drafts_and_forked_states_of_the_recurrence():
    """A step of four tokens a request leaves a state behind each; the accepted number picks the one that the next step
    starts from, and a copied slot is a fork of the request."""
    from chunked_gated_delta_kda_gb300 import binding
    from chunked_gated_delta_kda_gb300.inputs import make_decode_inputs
    N, S, H, V = 5, 3, 2, 300
    x = make_decode_inputs(N, H, S + 1 + 2, pool_slots=40, seed=31)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    part = lambda a, b: [d[k][:, a:b].contiguous() for k in ("q", "k", "v", "g", "beta")]  # noqa: E731
    base = torch.arange(N, dtype=torch.int32, device="cuda")[:, None] * (S + 1)
    slots = base + torch.arange(S + 1, dtype=torch.int32, device="cuda")
    pool = d["pool"][:40].clone()
    start = pool.clone()
    binding.fused_recurrent(*part(0, S + 1), pool, slots, num_accepted_tokens=torch.ones(N, dtype=torch.int32, device="cuda"))
    tokens, target, u, draft = draft_inputs(N, S, V, F32, seed=32)
    u[0, :S] = 0.0                                       # all accepted
    target[1, 0, tokens[1, 0]] = 0.0                     # none
    _, accepted = verify(tokens.cuda(), target.cuda(), u.cuda(), draft.cuda())
    assert accepted[0] == S + 1 and accepted[1] == 1
    forks = torch.stack([slots.gather(1, accepted[:, None].long() - 1)[:, 0], 20 + torch.arange(N, dtype=torch.int32, device="cuda")], 1)
    pages().page_copy(pool, forks)
    ahead = lambda p, s, n: binding.fused_recurrent(*part(S + 1, S + 3), p, s, num_accepted_tokens=n)  # noqa: E731
    of_forks = ahead(pool, torch.stack([forks[:, 1], forks[:, 1] + 10], 1), torch.ones_like(accepted))
    of_requests = ahead(pool, slots, accepted)
    assert torch.equal(of_forks, of_requests)
    for n, count in enumerate(accepted.tolist()):
        one = start.clone()
        slot = torch.full((N, 1), -1, dtype=torch.int32, device="cuda")
        slot[n] = slots[n, 0]
        for t in [*range(count), S + 1, S + 2]:
            o = binding.fused_recurrent(*part(t, t + 1), one, slot)
            if t > S:
                # (four tokens a window sum in another order than one: a rounding of o each)
                a, b = of_requests[n, t - S - 1].float(), o[n, 0].float()
                assert (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()
