"""Latent attention, its cache and its tables on the GPU against the 64-bit
oracle (``oracle.latent``), element by element within the oracle's bound of
what the types' roundings and 32-bit sums may add."""

import pytest
import torch

from oracle import latent as ol

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, FP: 2.0 ** -11}
TINY = {BF: 0.0, FP: 2.0 ** -25}


def api():
    from chunked_gated_delta_kda_gb300 import latent
    return latent


def near(got, want, err, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    inf = torch.isinf(want)
    assert torch.equal(inf, torch.isinf(got)) and torch.equal(want[inf], got[inf]), what
    off = ((got - want).abs() - err)[~inf]
    assert torch.isfinite(got[~inf]).all() and (off <= 0).all(), (what, off.max().item())


def cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def expanded(lens_q, lens_k, H, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, kv = (r(sum(lens_q), H, 192) * size).to(dtype), r(sum(lens_k), H, 256).to(dtype)
    return q, kv, r(sum(lens_k), 64).to(dtype), r(sum(lens_q), H, 128).to(dtype)


def run_fwd(q, kv, pe, lens_q, lens_k, causal=True, **kw):
    o, lse = api().latent_fwd(q[None].cuda(), kv[None].cuda(), pe[None].cuda(), causal=causal, cu_seqlens_q=cu(lens_q),
                              cu_seqlens_k=cu(lens_k), **kw)
    return o[0], lse[0]


CASES = [
    # queries, keys, heads, type, causal
    ([1], [1], 1, BF, True),
    ([37], [37], 3, BF, True),
    ([128], [128], 1, FP, False),
    ([129], [129], 2, BF, True),
    ([256, 257], [256, 257], 2, FP, True),
    ([64, 65, 1], [127, 128, 300], 2, BF, True),          # prefixes; one token behind 299
    ([1, 0, 3, 130], [2, 5, 0, 10], 2, BF, False),        # sequences without queries, without keys
    ([300, 5], [100, 1], 2, BF, True),                    # more queries than keys: rows that see nothing
    ([700], [900], 1, BF, True),
    ([513], [1100], 1, FP, False),
    ([300, 40], [4100, 3], 2, BF, True),                  # few queries on many keys: keys shared by four CTAs,
    ([5], [2300], 1, FP, False),
    ([300], [2100], 30, BF, True),                        # by two
]


@pytest.mark.parametrize("lens_q,lens_k,H,dtype,causal", CASES)
def test_fwd(lens_q, lens_k, H, dtype, causal):
    q, kv, pe, _ = expanded(lens_q, lens_k, H, dtype, seed=sum(lens_q))
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, causal)
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, lens_q, lens_k, causal, u=U[dtype], tiny=TINY[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


@pytest.mark.parametrize("lens_q,lens_k,H,dtype,causal", CASES)
def test_bwd(lens_q, lens_k, H, dtype, causal):
    q, kv, pe, do = expanded(lens_q, lens_k, H, dtype, seed=sum(lens_q))
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, causal)
    got = api().latent_bwd(q[None].cuda(), kv[None].cuda(), pe[None].cuda(), o[None], lse[None], do[None].cuda(),
                           causal=causal, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
    want = ol.latent_bwd(q, kv, pe, do, lens_q, lens_k, causal, u=U[dtype], tiny=TINY[dtype])
    for g, w, e, name in zip(got, want[:3], want[3:], ("dq", "dkv", "dk_pe")):
        near(g[0], w, e, name)


SHARED = [
    # one sequence with many more keys than the others: CTAs chosen on the device share its pairs
    ([300, 1, 0, 40, 5], [9000, 10, 7, 64, 1], 2, BF, True),
    ([1, 20, 600, 3, 3], [2, 8300, 500, 0, 3], 3, FP, False),
    ([700, 130, 1, 1, 9], [5000, 3200, 40, 1, 4], 5, BF, True),   # two of them, several pairs
    ([9000, 1, 1, 1, 1], [8500, 1, 1, 1, 1], 1, BF, True),        # more queries than keys; 36 pairs
    ([2, 2, 2, 2, 2], [1700] * 5, 30, FP, True),                  # none stands out: nothing is shared
]


@pytest.mark.parametrize("lens_q,lens_k,H,dtype,causal", SHARED)
def test_fwd_shared_keys(lens_q, lens_k, H, dtype, causal):
    assert api().latent_fwd_workspace_bytes(1, sum(lens_q), sum(lens_k), H, len(lens_q)) > 256
    q, kv, pe, _ = expanded(lens_q, lens_k, H, dtype, seed=sum(lens_q))
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, causal)
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, lens_q, lens_k, causal, u=U[dtype], tiny=TINY[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")      # too small to share anything
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, causal, workspace=ws)
    near(o, ro, eo, "o, not shared")
    near(lse, rl, el, "lse, not shared")


def test_fwd_shared_keys_are_contained_and_reported():
    """Bad rows of other sequences, peaked scores, a used workspace, equal bits, graphs, bad offsets, waits."""
    from chunked_gated_delta_kda_gb300 import binding
    lens_q, lens_k, H = [260, 30, 1, 70, 4], [8200, 100, 50, 70, 300], 2
    q, kv, pe, _ = expanded(lens_q, lens_k, H, BF, seed=20, size=8.0)
    want = ol.latent_fwd(q, kv, pe, lens_q, lens_k, u=U[BF])
    size = api().latent_fwd_workspace_bytes(1, sum(lens_q), sum(lens_k), H, 5)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever a part is not written
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, workspace=ws)
    assert binding.get_status(ws) == 0
    near(o, want[0], want[2], "o")
    near(lse, want[1], want[3], "lse")
    bad = kv.clone()
    bad[8200:8300] = float("nan")                                       # the second sequence's
    again = run_fwd(q, bad, pe, lens_q, lens_k, workspace=ws)
    rest = torch.tensor([i for i in range(sum(lens_q)) if not 260 <= i < 290], device="cuda")
    assert torch.equal(again[0][rest], o[rest]) and torch.equal(again[1][rest], lse[rest])

    dev = [t[None].cuda() for t in (q, kv, pe)]
    cq, ck, graph = cu(lens_q), cu(lens_k), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = api().latent_fwd(*dev, cu_seqlens_q=cq, cu_seqlens_k=ck, workspace=ws)
    ws.fill_(255)
    graph.replay()
    assert torch.equal(go[0], o) and torch.equal(gl[0], lse)
    ck.copy_(cu([100, 8200, 50, 70, 300]))                              # another sequence is the long one
    graph.replay()
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, lens_q, [100, 8200, 50, 70, 300], u=U[BF])
    near(go[0], ro, eo, "o, other lengths")
    near(gl[0], rl, el, "lse, other lengths")

    api().latent_fwd(*dev, cu_seqlens_q=cq, cu_seqlens_k=ck + 1, workspace=ws)
    assert binding.get_status(ws) == 4
    binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 1)
    try:
        api().latent_fwd(*dev, cu_seqlens_q=cq, cu_seqlens_k=ck, workspace=ws)
        assert binding.get_status(ws) == 5
    finally:
        binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 0)
    graph.replay()
    assert binding.get_status(ws) == 0
    near(go[0], ro, eo, "o, after a timeout")


@pytest.mark.parametrize("size,scale", [(20.0, None), (1.0, 0.5), (0.01, None)])
def test_fwd_peaked_and_flat_rows(size, scale):
    """Scores far apart (the running maximum moves often) and all alike."""
    lens = [300, 200]
    q, kv, pe, _ = expanded(lens, lens, 2, BF, seed=7, size=size)
    o, lse = run_fwd(q, kv, pe, lens, lens, scale=scale)
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, lens, lens, scale=scale, u=U[BF])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


def test_fixed_length_is_the_packed_result():
    q, kv, pe, do = expanded([200, 200], [200, 200], 3, BF, seed=8)
    o, lse = run_fwd(q, kv, pe, [200, 200], [200, 200])
    two = lambda t: t.view(2, 200, *t.shape[1:]).cuda()  # noqa: E731
    of, lf = api().latent_fwd(two(q), two(kv), two(pe))
    assert torch.equal(of.view_as(o), o) and torch.equal(lf.view_as(lse), lse)
    a = api().latent_bwd(two(q), two(kv), two(pe), of, lf, two(do))
    c = cu([200, 200])
    b = api().latent_bwd(q[None].cuda(), kv[None].cuda(), pe[None].cuda(), o[None], lse[None], do[None].cuda(),
                         cu_seqlens_q=c, cu_seqlens_k=c)
    for x, y in zip(a, b):
        assert torch.equal(x.reshape(y.shape), y)


def test_views_and_strides():
    """k_pe in place inside wider rows; views that start off a 16-byte boundary and transposed ones are copied."""
    q, kv, pe, do = (t.cuda() for t in expanded([150], [150], 2, BF, seed=9))
    o, lse = api().latent_fwd(q[None], kv[None], pe[None])
    wide = torch.full((1, 150, 576), float("nan"), dtype=BF, device="cuda")
    wide[..., 512:] = pe
    off = torch.zeros(150 * 64 + 1, dtype=BF, device="cuda")
    off[1:] = pe.flatten()
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)[None]
    for q2, pe2 in ((q[None], wide[..., 512:]), (q[None], off[1:].view(1, 150, 64)), (qt, pe[None])):
        o2, lse2 = api().latent_fwd(q2, kv[None], pe2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        a, b = (api().latent_bwd(x, kv[None], y, o, lse, do[None]) for x, y in ((q[None], pe[None]), (q2, pe2)))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_never_reach_a_result(bad):
    lens_q, lens_k = [70, 90, 130], [70, 90, 130]
    q, kv, pe, do = expanded(lens_q, lens_k, 2, BF, seed=10)
    runs = []
    for fill in (None, bad):
        x = [t.clone() for t in (q, kv, pe, do)]
        if fill is not None:
            for t in x:
                t[:70] = fill
                t[160:] = fill
        o, lse = run_fwd(*x[:3], lens_q, lens_k)
        g = api().latent_bwd(*(t[None].cuda() for t in x[:3]), o[None], lse[None], x[3][None].cuda(),
                             cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
        runs.append([o[70:160], lse[70:160]] + [t[0, 70:160] for t in g])
    for a, b in zip(*runs):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_bwd_equal_inputs_give_equal_bits():
    q, kv, pe, do = (t[None].cuda() for t in expanded([1000], [1000], 4, BF, seed=11))
    o, lse = api().latent_fwd(q, kv, pe)
    a, b = (api().latent_bwd(q, kv, pe, o, lse, do) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_empty_sides():
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    o, lse = api().latent_fwd(z(2, 3, 2, 192), z(2, 0, 2, 256), z(2, 0, 64))
    assert (o == 0).all() and torch.isinf(lse).all()
    dq, dkv, dpe = api().latent_bwd(z(2, 3, 2, 192), z(2, 0, 2, 256), z(2, 0, 64), o, lse, o)
    assert (dq == 0).all() and dkv.numel() == 0 and dpe.numel() == 0
    o, lse = api().latent_fwd(z(2, 0, 2, 192), z(2, 3, 2, 256), z(2, 3, 64))
    assert o.numel() == 0 and lse.numel() == 0
    dq, dkv, dpe = api().latent_bwd(z(2, 0, 2, 192), z(2, 3, 2, 256), z(2, 3, 64), o, lse, o)
    assert dq.numel() == 0 and (dkv == 0).all() and (dpe == 0).all()


def test_bad_offsets_are_reported():
    from chunked_gated_delta_kda_gb300 import binding
    q, kv, pe, do = (t[None].cuda() for t in expanded([20], [20], 1, BF))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    good, short = cu([20]), torch.tensor([0, 19], dtype=torch.int32, device="cuda")
    o, lse = api().latent_fwd(q, kv, pe, cu_seqlens_q=good, cu_seqlens_k=good, workspace=ws)
    assert binding.get_status(ws) == 0
    down = torch.tensor([0, 15, 12, 20], dtype=torch.int32, device="cuda")
    for a, b in ((short, good), (good, short), (down, down)):
        api().latent_fwd(q, kv, pe, cu_seqlens_q=a, cu_seqlens_k=b, workspace=ws)
        assert binding.get_status(ws) == 4
    wb = torch.zeros(api().latent_bwd_workspace_bytes(1, 20, 20, 1, 3), dtype=torch.uint8, device="cuda")
    api().latent_bwd(q, kv, pe, o, lse, do, cu_seqlens_q=down, cu_seqlens_k=down, workspace=wb)
    assert binding.get_status(wb) == 4


# ---------------------------------------------------------------------------
def paged(lens, page, dtype, seed=0, extra=2, fill=None):
    """A cache with the sequences' rows on shuffled pages, its table, and (fill) every other row filled with it."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(l, 0) // page) for l in lens]
    total, width = sum(need) + extra, max(1, max(need))
    cache = torch.randn(total, page, 576, generator=g).to(dtype)
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    used = torch.zeros(total, page, dtype=torch.bool)
    for i, l in enumerate(lens):
        for j in range(need[i]):
            table[i, j] = order.pop()
            used[table[i, j], :min(page, l - j * page)] = True
    if fill is not None:
        cache[~used] = fill
    return cache, table


DECODE = [
    # lengths, tokens, heads, page, type
    ([1], 1, 1, 16, BF),
    ([64], 1, 16, 64, BF),
    ([65, 0, 1, 63], 1, 17, 16, BF),
    ([200, 129], 1, 32, 32, FP),
    ([333, 3, 0, 1000], 4, 16, 64, BF),                   # more tokens than rows: some see nothing
    ([500], 1, 64, 128, FP),
    ([300, 77], 1, 65, 192, BF),                          # two blocks of rows, the second with one
    ([130], 2, 64, 16, BF),
    ([40] * 70, 1, 8, 16, BF),                            # short sequences, several a CTA
    ([9000], 3, 5, 64, FP),                               # one long sequence over the whole GPU
    ([70] + [0] * 100 + [1000, 0, 5] + [0] * 33 + [64] + [0] * 40, 1, 20, 64, BF),   # padded entries between and behind
    ([0, 0, 0], 2, 3, 16, FP),
]


@pytest.mark.parametrize("lens,S,H,page,dtype", DECODE)
def test_decode(lens, S, H, page, dtype):
    cache, table = paged(lens, page, dtype, seed=len(lens), fill=float("nan"))
    q = torch.randn(len(lens), S, H, 576, generator=torch.Generator().manual_seed(1)).to(dtype)
    n = torch.tensor(lens, dtype=torch.int32)
    o, lse = api().latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda())
    ro, rl, eo, el = ol.latent_decode(q, cache, table, n, u=U[dtype], tiny=TINY[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


def test_decode_peaked_scores():
    cache, table = paged([700, 90], 64, BF, seed=3)
    q = (torch.randn(2, 1, 32, 576, generator=torch.Generator().manual_seed(2)) * 12).to(BF)
    n = torch.tensor([700, 90], dtype=torch.int32)
    o, lse = api().latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), scale=0.2)
    ro, rl, eo, el = ol.latent_decode(q, cache, table, n, scale=0.2, u=U[BF])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


@pytest.mark.parametrize("page", [16, 64])
def test_decode_missing_pages_and_bad_lengths(page):
    from chunked_gated_delta_kda_gb300 import binding
    lens = [300, 100, 200]
    cache, table = paged(lens, page, BF, seed=5)
    cache[:, 3] = float("nan") if page == 16 else cache[:, 3]
    cache = torch.nan_to_num(cache, nan=0.5)
    table[0, 1], table[2, 0], table[2, 2] = -7, cache.shape[0], 1 << 30
    n = torch.tensor([300, -5, 10 ** 6], dtype=torch.int32)
    q = torch.randn(3, 2, 8, 576, generator=torch.Generator().manual_seed(4)).to(BF)
    ws = torch.full((api().latent_decode_workspace_bytes(3, 2, 8),), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = api().latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), workspace=ws)
    assert binding.get_status(ws) == 8
    ro, rl, eo, el = ol.latent_decode(q, cache, table, n, u=U[BF])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")
    good = torch.tensor([1, 1, 1], dtype=torch.int32)
    table[2, 0] = 0
    api().latent_decode(q.cuda(), cache.cuda(), table.cuda(), good.cuda(), workspace=ws)
    assert binding.get_status(ws) == 0


def test_decode_and_append_past_32_bit_offsets():
    """A cache of more than 2^31 elements: its last pages."""
    page, pages = 64, (1 << 31) // (576 * 64) + 60
    cache = torch.empty(pages, page, 576, dtype=BF, device="cuda")
    lens, width = [150], 3
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32)
    rows = torch.randn(150, 576, generator=torch.Generator().manual_seed(6)).to(BF)
    at = torch.arange(150)
    slots = table[0][at // page].long() * page + at % page
    api().latent_append(rows.cuda(), slots.cuda(), cache)
    assert torch.equal(cache.view(-1, 576)[slots.cuda()].cpu(), rows)
    q = torch.randn(1, 1, 16, 576, generator=torch.Generator().manual_seed(7)).to(BF)
    n = torch.tensor(lens, dtype=torch.int32)
    o, lse = api().latent_decode(q.cuda(), cache, table.cuda(), n.cuda())
    small = torch.zeros(width, page, 576, dtype=BF)
    small.view(-1, 576)[:150] = rows
    ro, rl, eo, el = ol.latent_decode(q, small, torch.arange(width)[None], n, u=U[BF])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,page,dtype,norm", [(1, 16, BF, True), (5, 64, FP, True), (333, 16, BF, False), (1000, 48, FP, True)])
def test_append(T, page, dtype, norm):
    from chunked_gated_delta_kda_gb300 import binding
    g = torch.Generator().manual_seed(T)
    pages = T // page + 3
    wide = (torch.randn(T, 640, generator=g) * 3).to(dtype)
    rows = wide[:, 8:584]                                 # rows of a wider tensor, 16-byte aligned
    cache = torch.randn(pages, page, 576, generator=g).to(dtype)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::7] = -1
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(dtype) if norm else None
    want = ol.latent_append(rows, slots, cache, weight, 1e-5)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (slots.cuda(),), dict(norm_weight=None if weight is None else weight.cuda(), eps=1e-5, workspace=ws)
    got = api().latent_append(wide.cuda()[:, 8:584], *args[0], cache.cuda(), **args[1])
    # 512 squares in 32 bits, a reciprocal square root and two products, then the type
    near(got, want, (U[dtype] + 520 * 2.0 ** -24) * want.abs() + TINY[dtype] if norm else torch.zeros_like(want), "cache")
    assert binding.get_status(ws) == 0
    got2 = api().latent_append(wide.cuda()[:, 3:579], *args[0], cache.cuda(), **args[1])   # off the boundary: copied
    want2 = ol.latent_append(wide[:, 3:579], slots, cache, weight, 1e-5)
    near(got2, want2, (U[dtype] + 520 * 2.0 ** -24) * want2.abs() + TINY[dtype] if norm else torch.zeros_like(want2), "cache")


def test_append_of_one_row_takes_any_row_step():
    """The step between rows means nothing where there is one row."""
    for wide in (577, 580, 584, 1152):
        rows = torch.randn(1, wide, generator=torch.Generator().manual_seed(wide)).to(BF).cuda()[:, :576]
        cache = torch.zeros(1, 16, 576, dtype=BF, device="cuda")
        api().latent_append(rows, torch.tensor([3], device="cuda"), cache)
        assert torch.equal(cache[0, 3], rows[0]) and int(cache.count_nonzero()) == int(rows.count_nonzero())


def test_workspaces_elsewhere_are_refused():
    q, kv, pe, do = (t[None].cuda() for t in expanded([3], [3], 1, BF, seed=18))
    cache, table = (t.cuda() for t in paged([3], 16, BF, seed=19))
    lens, host = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.zeros(1 << 22, dtype=torch.uint8)
    o, lse = api().latent_fwd(q, kv, pe)
    slot = torch.tensor([0], device="cuda")
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    for call in (lambda w: api().latent_fwd(q, kv, pe, workspace=w),
                 lambda w: api().latent_bwd(q, kv, pe, o, lse, do, workspace=w),
                 lambda w: api().latent_decode(cache[:1, None, :1], cache, table, lens, workspace=w),
                 lambda w: api().latent_append(cache[0, :1], slot, cache, workspace=w),
                 lambda w: api().block_tables(lens, one, table, one, one, 16, 1, workspace=w)):
        for bad in (host, host.cuda()[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)


def test_append_refuses_slots_past_the_cache():
    from chunked_gated_delta_kda_gb300 import binding
    cache = torch.zeros(2, 16, 576, dtype=BF, device="cuda")
    rows = torch.ones(3, 576, dtype=BF, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    api().latent_append(rows, torch.tensor([0, 32, 1 << 40], device="cuda"), cache, workspace=ws)
    assert binding.get_status(ws) == 8
    assert (cache[0, 0] == 1).all() and cache.view(-1, 576)[1:].abs().sum() == 0
    api().latent_append(rows[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), cache, workspace=ws)
    assert binding.get_status(ws) == 0


# ---------------------------------------------------------------------------
def run_tables(lens, new, table, free, head, page, tokens):
    from chunked_gated_delta_kda_gb300 import binding
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t = i(table).reshape(len(lens), -1)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    slots, c, out, h = api().block_tables(i(lens), i(new), t, i(free), i([head]), page, tokens, workspace=ws)
    return (slots.tolist(), c.tolist(), out.tolist(), h.item(), t.tolist()), binding.get_status(ws)


@pytest.mark.parametrize("n,page,longest,most,head,pad", [
    (1, 16, 0, 1, 0, 0), (7, 16, 100, 60, 3, 5), (300, 64, 500, 1, 0, 0), (2500, 16, 64, 20, 11, 3), (3, 128, 5, 20000, 0, 0),
    (5000, 1, 3, 2, 2, 0)])
def test_tables(n, page, longest, most, head, pad):
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, longest + 1, (n,), generator=g).tolist()
    new = torch.randint(0, most + 1, (n,), generator=g).tolist()
    held = [-(-l // page) for l in lens]
    width = max(-(-(l + b) // page) for l, b in zip(lens, new)) + 1
    order = torch.randperm(sum(held) + sum(-(-(l + b) // page) for l, b in zip(lens, new)) + head, generator=g).tolist()
    table = [[order.pop() for _ in range(k)] + [-1] * (width - k) for k in held]
    want = ol.block_tables(lens, new, table, order, head, page, sum(new) + pad)
    got, status = run_tables(lens, new, table, order, head, page, sum(new) + pad)
    assert status == 0 and got == tuple(want)


@pytest.mark.parametrize("case", [
    dict(lens=[3, 0, 9], new=[5, 40, 2], width=3, free=[9, 8], head=0, page=4, tokens=47),        # too few pages, too narrow
    dict(lens=[-2, 5], new=[3, -1], width=4, free=[1, 2, 3], head=0, page=4, tokens=3),           # negative lengths
    dict(lens=[0, 0], new=[6, 6], width=4, free=[1, 2, 3, 4, 5, 6], head=1, page=4, tokens=7),    # more tokens than the map
    dict(lens=[0], new=[2], width=1, free=[4], head=-1, page=4, tokens=2),                        # a head outside the list
    dict(lens=[2], new=[1], width=1, free=[], head=0, page=4, tokens=1),                          # a held cell without a page
])
def test_tables_faults_are_reported_and_contained(case):
    width = case.pop("width")
    table = [[-1] * width if len(case["lens"]) == 1 else [20 + 4 * i + j if j * case["page"] < l else -1 for j in range(width)]
             for i, l in enumerate(case["lens"])]
    want = ol.block_tables(case["lens"], case["new"], table, case["free"], case["head"], case["page"], case["tokens"])
    got, status = run_tables(case["lens"], case["new"], table, case["free"], case["head"], case["page"], case["tokens"])
    assert status == 8 and got == tuple(want)


# ---------------------------------------------------------------------------
def test_other_streams_and_graphs():
    """Every operator on a stream of its own and captured into a graph that is replayed on new contents."""
    q, kv, pe, do = (t[None].cuda() for t in expanded([200], [200], 2, BF, seed=12))
    cache, table = (t.cuda() for t in paged([130, 40], 64, BF, seed=13))
    lens = torch.tensor([130, 40], dtype=torch.int32, device="cuda")
    qd = torch.randn(2, 1, 16, 576, generator=torch.Generator().manual_seed(14)).to(BF).cuda()
    rows, slots = torch.ones(2, 576, dtype=BF, device="cuda"), torch.tensor([1, 70], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    new, free, head, tab = torch.ones(2, **i32), torch.arange(9, **i32), torch.zeros(1, **i32), torch.zeros(2, 8, **i32)

    def everything():
        o, lse = api().latent_fwd(q, kv, pe)
        g = api().latent_bwd(q, kv, pe, o, lse, do)
        c = api().latent_append(rows, slots, cache)
        d = api().latent_decode(qd, c, table, lens)
        t = api().block_tables(lens, new, tab, free, head, 16, 4)
        return (o, lse) + g + d + t

    want = [t.clone() for t in everything()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = everything()
        q.mul_(0.5)
        qd.mul_(0.5)
        graph.replay()
        side.synchronize()
    want = everything()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_waits_that_run_out_are_reported():
    """With one poll a wait every role gives up: the calls end by themselves with KDA_ERR_TIMEOUT, and the next
    ones are right."""
    from chunked_gated_delta_kda_gb300 import binding
    q, kv, pe, do = (t[None].cuda() for t in expanded([600], [600], 2, BF, seed=15))
    cache, table = (t.cuda() for t in paged([900], 64, BF, seed=16))
    lens = torch.tensor([900], dtype=torch.int32, device="cuda")
    qd = torch.randn(1, 1, 16, 576, generator=torch.Generator().manual_seed(17)).to(BF).cuda()
    ws = torch.zeros(api().latent_bwd_workspace_bytes(1, 600, 600, 2, 1), dtype=torch.uint8, device="cuda")
    wd = torch.zeros(api().latent_decode_workspace_bytes(1, 1, 16), dtype=torch.uint8, device="cuda")

    def calls():
        o, lse = api().latent_fwd(q, kv, pe, workspace=ws)
        status = [binding.get_status(ws)]
        g = api().latent_bwd(q, kv, pe, o, lse, do, workspace=ws)
        status.append(binding.get_status(ws))
        d = api().latent_decode(qd, cache, table, lens, workspace=wd)
        status.append(binding.get_status(wd))
        return (o, lse) + g + d, status

    want, status = calls()
    assert status == [0, 0, 0]
    binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 1)
    try:
        assert calls()[1] == [5, 5, 5]
    finally:
        binding.debug_set(binding.KDA_DEBUG_WAIT_LIMIT, 0)
    got, status = calls()
    assert status == [0, 0, 0] and all(torch.equal(a, b) for a, b in zip(want, got))


def test_serving_layer():
    """Prefill, tables, cache and absorbed decode agree with the expanded form over whole sequences.  Query and
    output of the absorbed form, the expanded keys, values and output are each rounded to bf16 (2^-8 of themselves),
    and the two forms' weights besides: six roundings, against the norm."""
    from chunked_gated_delta_kda_gb300 import latent_serving
    assert latent_serving.main() < 6 * 2.0 ** -8


def test_training_layer():
    """The gradient of the layer's input against a difference quotient along a direction, in 64 bits."""
    from chunked_gated_delta_kda_gb300.latent_serving import LatentLayer
    g = torch.Generator(device="cuda").manual_seed(2)
    layer = LatentLayer(256, 2, 1, pages=1)
    x = torch.randn(1, 96, 256, generator=g, device="cuda").to(BF)
    grad = torch.randn(1, 96, 2, 128, generator=g, device="cuda").to(BF)
    o, dx = layer.train(x, grad)
    step = torch.randn(1, 96, 256, generator=g, device="cuda", dtype=torch.float64)

    def loss(x):
        q = (x @ layer.w_q.double().T).view(96, 2, 192)
        rows = x @ layer.w_row.double().T
        kv = torch.einsum("tc,hdc->thd", rows[0, :, :512], layer.w_up.double())
        out = ol.latent_fwd(q.cpu(), kv.cpu(), rows[0, :, 512:].cpu(), [96], [96])[0]
        return (out * grad[0].double().cpu()).sum()

    e = 2.0 ** -8
    diff = (loss(x.double() + e * step) - loss(x.double() - e * step)) / (2 * e)
    got = (dx.double() * step).sum().cpu()
    # sums of 96 * 256 terms with independent signs: a few bf16 roundings of dx's norm times the step's rms (1)
    assert (diff - got).abs() <= 8 * 2.0 ** -8 * dx.double().norm().cpu(), (diff, got)


# ---------------------------------------------------------------------------
# fp16 gradients: dS = P (dP - D) is as small as dout times the weights, or larger than fp16 holds.  A small scale of
# the queries and keys (and a large one of the scores) makes dq and dk large beside dS, so that their own rounding to
# fp16 does not hide dS's.
HALF_GRADS = [
    # lengths, size of dout of each (sequence, head), of the values, of queries and keys, scale
    ([2048], [[2.0 ** -16]], 1.0, 2.0 ** -6, 2.0 ** 12 * 192 ** -0.5),
    ([2048], [[2.0 ** -20]], 1.0, 2.0 ** -7, 2.0 ** 14 * 192 ** -0.5),
    ([600, 2048, 1], [[2.0 ** 8] * 2, [2.0 ** -16] * 2, [1.0] * 2], 1.0, 2.0 ** -6, 2.0 ** 12 * 192 ** -0.5),   # sequences apart
    ([700], [[2.0 ** 6, 2.0 ** -17]], 1.0, 2.0 ** -6, 2.0 ** 12 * 192 ** -0.5),                                 # heads apart
    ([1, 2, 3], [[2.0 ** -10] * 40] * 3, 1.0, 2.0 ** -3, 2.0 ** 6 * 192 ** -0.5),     # more heads than a row's pairs
    ([300], [[2.0 ** 12]], 2.0 ** 4, 2.0 ** -6, None),                                # dS beyond 65504
    ([300], [[2.0 ** -12]], 2.0 ** 11, 1.0, None),                                    # large values
]


@pytest.mark.parametrize("lens,sizes,size_v,size_x,scale", HALF_GRADS)
def test_bwd_fp16_gradients_of_any_size(lens, sizes, size_v, size_x, scale):
    H = len(sizes[0])
    q, kv, pe, do = (t.float() for t in expanded(lens, lens, H, torch.float32, seed=21))
    for i, row in enumerate(sizes):
        for h, size in enumerate(row):
            do[sum(lens[:i]):sum(lens[:i + 1]), h] *= size
    kv[..., :128] *= size_x
    kv[..., 128:] *= size_v
    q, kv, pe, do = (q * size_x).to(FP), kv.to(FP), (pe * size_x).to(FP), do.to(FP)
    o, lse, parts = ol.latent_bwd_norms(q, kv, pe, do, lens, lens, scale, u=U[FP], tiny=TINY[FP])
    dq, dkv, dpe = (t[0].double().cpu() for t in api().latent_bwd(
        q[None].cuda(), kv[None].cuda(), pe[None].cuda(), o.to(FP)[None].cuda(), lse.float()[None].cuda(), do[None].cuda(),
        scale=scale, cu_seqlens_q=cu(lens), cu_seqlens_k=cu(lens)))
    for part in parts:
        for name, (rows, h, channels, want, bound) in part.items():
            got = {"dq": dq, "dk": dkv, "dv": dkv, "dpe": dpe}[name]
            got = got[rows, channels] if h is None else got[rows, h, channels]
            off = torch.linalg.matrix_norm(got - want).item()
            assert off <= bound, (name, rows, h, off, bound)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 6e4])
def test_other_sequences_never_reach_an_fp16_gradient(bad):
    """Nor through the factor that dS carries; and rows that see no key, whatever their dout, do not choose it."""
    lens_q, lens_k, runs = [70, 90, 130], [70, 60, 130], []
    q, kv, pe, do = expanded(lens_q, lens_k, 2, FP, seed=22)
    do = do * 2.0 ** -10
    for fill in (None, bad):
        x = [t.clone() for t in (q, kv, pe, do)]
        if fill is not None:
            for t, keys in zip(x, (False, True, True, False)):
                t[:70] = fill
                t[130 if keys else 160:] = fill
            x[3][70:100] = 6e4
        o, lse = run_fwd(*x[:3], lens_q, lens_k)
        g = api().latent_bwd(*(t[None].cuda() for t in x[:3]), o[None], lse[None], x[3][None].cuda(),
                             cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
        runs.append([g[0][0, 70:160], g[1][0, 70:130], g[2][0, 70:130]])
    for a, b in zip(*runs):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_serving_layer_without_room_says_so():
    """A token without a page, in the free list or in the table, or rows that do not match the lengths: an error in
    place of another row's keys, and the layer goes on as if the step had not been."""
    from chunked_gated_delta_kda_gb300 import binding
    from chunked_gated_delta_kda_gb300.latent_serving import LatentLayer
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(200, 128, generator=g, device="cuda").to(BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for room in (dict(pages=3, width=8), dict(pages=8, width=1)):
        layer, fresh = (LatentLayer(128, 2, 2, page_size=64, **room) for _ in range(2))
        with pytest.raises(binding.KdaError) as e:
            layer.prefill(x, i32(150, 50))
        assert e.value.code == 8
        with pytest.raises(ValueError, match="rows"):
            layer.prefill(x[:70], i32(40, 20))
        assert layer.lens.tolist() == [0, 0] and layer.head.item() == 0 and layer.cache.count_nonzero() == 0
        assert torch.equal(layer.prefill(x[:127], i32(64, 63)), fresh.prefill(x[:127], i32(64, 63)))
        with pytest.raises(binding.KdaError):
            for _ in range(80):
                layer.decode(x[:2])
        assert layer.lens.tolist() == ([64, 63] if room["width"] == 1 else [65, 64])


@pytest.mark.parametrize("size,dtype", [(256, torch.uint8), (1000, torch.uint8), (64, torch.float32)])
def test_a_workspace_that_is_too_small_still_gets_the_status(size, dtype):
    """The calls use another one beside it; what they record must not stay there."""
    from chunked_gated_delta_kda_gb300 import binding
    ws = torch.zeros(size, dtype=dtype, device="cuda")
    cache, table = (t.cuda() for t in paged([40], 16, BF, seed=23))
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    qd = torch.randn(1, 1, 4, 576, generator=torch.Generator().manual_seed(24)).to(BF).cuda()
    want = api().latent_decode(qd, cache, table, n)
    for lens, status in ((n, 0), (n + 9, 8), (n, 0)):   # a fault, and none again
        got = api().latent_decode(qd, cache, table, lens, workspace=ws)
        assert binding.get_status(ws) == status
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, kv, pe, do = (t[None].cuda() for t in expanded([20], [20], 1, BF, seed=25))
    o, lse = api().latent_fwd(q, kv, pe)
    down = torch.tensor([0, 15, 12, 20], dtype=torch.int32, device="cuda")
    for c, status in ((cu([20]), 0), (down, 4), (cu([20]), 0)):
        api().latent_bwd(q, kv, pe, o, lse, do, cu_seqlens_q=c, cu_seqlens_k=c, workspace=ws)
        assert binding.get_status(ws) == status


# ---------------------------------------------------------------------------
def mixed(n, seed, empty=()):
    """n lengths around the tiles' borders, many of none or one, `empty` (a range) of none."""
    g = torch.Generator().manual_seed(seed)
    some = [0, 0, 1, 1, 2, 5, 63, 64, 65, 127, 128, 129, 130, 257]
    lens = [some[i] for i in torch.randint(0, len(some), (n,), generator=g).tolist()]
    return [0 if i in empty else l for i, l in enumerate(lens)]


def fwd_and_bwd(lens_q, lens_k, H, dtype, causal, seed):
    q, kv, pe, do = expanded(lens_q, lens_k, H, dtype, seed=seed)
    o, lse = run_fwd(q, kv, pe, lens_q, lens_k, causal)
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, lens_q, lens_k, causal, u=U[dtype], tiny=TINY[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")
    got = api().latent_bwd(q[None].cuda(), kv[None].cuda(), pe[None].cuda(), o[None], lse[None], do[None].cuda(),
                           causal=causal, cu_seqlens_q=cu(lens_q), cu_seqlens_k=cu(lens_k))
    want = ol.latent_bwd(q, kv, pe, do, lens_q, lens_k, causal, u=U[dtype], tiny=TINY[dtype])
    for g, w, e, name in zip(got, want[:3], want[3:], ("dq", "dkv", "dk_pe")):
        near(g[0], w, e, name)


@pytest.mark.parametrize("n,H,dtype,causal,empty", [
    (30, 2, BF, True, range(0)), (31, 2, FP, True, range(0, 4)), (32, 2, BF, False, range(28, 32)),
    (33, 1, FP, True, range(30, 33)), (70, 3, BF, True, range(27, 40)), (70, 2, FP, False, range(0, 33)),
    (257, 1, BF, True, range(100, 180))])
def test_many_packed_sequences(n, H, dtype, causal, empty):
    """Up to 31 sequences a tile finds its own by one vote, from 32 on by bisection."""
    fwd_and_bwd(mixed(n, n, empty), mixed(n, n + 1000, range(5, 8)), H, dtype, causal, n)


@pytest.mark.parametrize("n,long,dtype", [(31, 20, BF), (32, 0, FP), (70, 69, BF)])
def test_many_packed_sequences_that_share_keys(n, long, dtype):
    lens_q, lens_k = mixed(n, n, range(10, 14)), mixed(n, n + 1)
    lens_q[long], lens_k[long] = 300, 8300
    assert api().latent_fwd_workspace_bytes(1, sum(lens_q), sum(lens_k), 2, n) > 256
    fwd_and_bwd(lens_q, lens_k, 2, dtype, True, n)


@pytest.mark.parametrize("n,dtype", [(31, FP), (34, BF)])
def test_many_packed_sequences_in_clusters(n, dtype):
    """2048 keys a sequence on average, few queries: clusters."""
    lens_q = [l % 30 for l in mixed(n, n, range(6, 9))]
    lens_k = [0 if i % 7 == 3 else 2900 + 131 * (i % 5) for i in range(n)]
    assert sum(lens_k) >= 2048 * n and api().latent_fwd_workspace_bytes(1, sum(lens_q), sum(lens_k), 1, n) == 256
    fwd_and_bwd(lens_q, lens_k, 1, dtype, True, n)


@pytest.mark.parametrize("B,Tq,Tk,H,dtype,causal", [
    (3, 70, 200, 2, BF, True), (2, 300, 129, 2, FP, True), (4, 1, 65, 3, FP, False), (40, 33, 33, 1, FP, True),
    (1, 20, 4100, 2, BF, True), (2, 5, 2100, 3, FP, False)])             # the last two: clusters
def test_fixed_length(B, Tq, Tk, H, dtype, causal):
    q, kv, pe, do = expanded([Tq] * B, [Tk] * B, H, dtype, seed=B * Tk)
    lead = lambda t: t.view(B, -1, *t.shape[1:]).cuda()  # noqa: E731
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    o, lse = api().latent_fwd(lead(q), lead(kv), lead(pe), causal=causal)
    ro, rl, eo, el = ol.latent_fwd(q, kv, pe, [Tq] * B, [Tk] * B, causal, u=U[dtype], tiny=TINY[dtype])
    near(flat(o), ro, eo, "o")
    near(flat(lse), rl, el, "lse")
    got = api().latent_bwd(lead(q), lead(kv), lead(pe), o, lse, lead(do), causal=causal)
    want = ol.latent_bwd(q, kv, pe, do, [Tq] * B, [Tk] * B, causal, u=U[dtype], tiny=TINY[dtype])
    for g, w, e, name in zip(got, want[:3], want[3:], ("dq", "dkv", "dk_pe")):
        near(flat(g), w, e, name)


@pytest.mark.parametrize("page,S,H,dtype", [(16, 1, 4, BF), (32, 2, 16, FP), (64, 1, 64, BF), (128, 3, 5, FP)])
def test_decode_missing_pages_meet_what_the_tiles_before_left(page, S, H, dtype):
    """Rows that no token sees are NaN, each CTA walks some ten tiles, so the ring slots of rows on missing pages hold
    NaN of sequences before."""
    from chunked_gated_delta_kda_gb300 import binding
    g = torch.Generator().manual_seed(page)
    lens = torch.randint(1, 260, (600,), generator=g).tolist()
    cache, table = paged(lens, page, dtype, seed=page, fill=float("nan"))
    for i in range(0, 600, 2):                            # every other sequence misses pages, its first or last ones too
        cells = -(-lens[i] // page)
        for j in torch.randint(0, cells, (1 + i % 3,), generator=g).tolist():
            table[i, j] = (-1, cache.shape[0], 1 << 30)[i % 3]
    q = torch.randn(600, S, H, 576, generator=g).to(dtype)
    n = torch.tensor(lens, dtype=torch.int32)
    ws = torch.zeros(api().latent_decode_workspace_bytes(600, S, H), dtype=torch.uint8, device="cuda")
    o, lse = api().latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), workspace=ws)
    assert binding.get_status(ws) == 8
    ro, rl, eo, el = ol.latent_decode(q, cache, table, n, u=U[dtype], tiny=TINY[dtype])
    near(o, ro, eo, "o")
    near(lse, rl, el, "lse")


@pytest.mark.parametrize("H,more", [(2, 0), (60, 0), (2, 40), (1, 2 ** 17), (2, 9000)])
def test_offsets_that_step_back_are_reported(H, more):
    """Also where no tile of the sequence that steps back is looked up.  Few sequences and 40 more, few heads and many;
    2^17 more keys: clusters; 9000: CTAs that share keys."""
    from chunked_gated_delta_kda_gb300 import binding
    step, extra = [0, 600, 300, 900], [1] * {40: 40, 9000: 8}.get(more, 1)
    at_q = torch.tensor(step + [900 + i + 1 for i in range(len(extra))], dtype=torch.int32, device="cuda")
    tq, many = 900 + len(extra), more if more > 40 else 0
    at_k = at_q.clone()
    at_k[-1] += many
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    args = z(1, tq, H, 192), z(1, tq + many, H, 256), z(1, tq + many, 64)
    good_q, good_k = at_q.clone(), at_k.clone()
    good_q[1:3] = good_k[1:3] = 450
    ws = torch.zeros(max(256, api().latent_fwd_workspace_bytes(1, tq, tq + many, H, len(at_q) - 1)), dtype=torch.uint8, device="cuda")
    assert (ws.numel() > 256) == (more == 9000)
    wb = torch.zeros(api().latent_bwd_workspace_bytes(1, tq, tq + many, H, len(at_q) - 1), dtype=torch.uint8, device="cuda")
    for a, b, status in ((good_q, good_k, 0), (at_q, at_k, 4), (at_q, good_k, 4), (good_q, at_k, 4)):
        o, lse = api().latent_fwd(*args, cu_seqlens_q=a, cu_seqlens_k=b, workspace=ws)
        assert binding.get_status(ws) == status
        api().latent_bwd(*args, o, lse, o, cu_seqlens_q=a, cu_seqlens_k=b, workspace=wb)
        assert binding.get_status(wb) == status
    none = torch.zeros_like(at_q)
    o = z(1, 0, H, 128)
    api().latent_bwd(z(1, 0, H, 192), *args[1:], o, o[..., 0].float(), o, cu_seqlens_q=none, cu_seqlens_k=at_k, workspace=wb)
    assert binding.get_status(wb) == 4


def test_expanded_form_past_32_bit_offsets():
    """Packed tensors of more than 2^31 elements: the last sequences get the bits that they get alone."""
    lens, H = [200] * 660 + [129, 1, 270], 128
    T, last = sum(lens), 400
    assert T * H * 128 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(26)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    q, kv, pe, do = r(1, T, H, 192), r(1, T, H, 256), r(1, T, 64), r(1, T, H, 128)
    c, alone = cu(lens), cu(lens[-3:])
    o, lse = api().latent_fwd(q, kv, pe, cu_seqlens_q=c, cu_seqlens_k=c)
    grads = api().latent_bwd(q, kv, pe, o, lse, do, cu_seqlens_q=c, cu_seqlens_k=c)
    tail = [t[:, T - last:].contiguous() for t in (q, kv, pe, do)]
    o2, lse2 = api().latent_fwd(*tail[:3], cu_seqlens_q=alone, cu_seqlens_k=alone)
    assert torch.equal(o[:, T - last:], o2) and torch.equal(lse[:, T - last:], lse2)
    for x, y in zip(grads, api().latent_bwd(*tail[:3], o2, lse2, tail[3], cu_seqlens_q=alone, cu_seqlens_k=alone)):
        assert torch.equal(x[:, T - last:], y)


def test_serving_layer_prefills_new_requests_only():
    """A second prompt of a request would not see the first; other requests may be prefilled beside cached ones."""
    from chunked_gated_delta_kda_gb300.latent_serving import LatentLayer
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(90, 128, generator=g, device="cuda").to(BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    layer, fresh = (LatentLayer(128, 2, 2, pages=8, width=2) for _ in range(2))
    layer.prefill(x[:50], i32(50, 0))
    with pytest.raises(ValueError, match="cached"):
        layer.prefill(x[50:], i32(40, 0))
    assert layer.lens.tolist() == [50, 0]
    a, b = layer.prefill(x[50:], i32(0, 40)).float(), fresh.prefill(x, i32(50, 40))[50:].float()
    # the projections of 40 and of 90 rows may sum in another order: a rounding of rows, keys, values and output each
    assert (a - b).norm() <= 4 * 2.0 ** -8 * b.norm()
