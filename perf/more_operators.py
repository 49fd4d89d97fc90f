"""Serving over the paged latent cache: the cases that are measured, and the operators' plain forms.

Requests whose tokens' latent rows are on pages of a cache are served in steps
of several tokens, share the pages of common prompts, and give pages back:

  chunk    attention of a chunk of new tokens a request over all its cached
           rows (the chunk's own included): keys and values are expanded from
           the paged rows [576] by the heads' up-projection [H, 256, 512];
           queries [T, H, 128 + 64], packed; output [T, H, 128], log-sum-exp.
  verify   drafted tokens against the target's probabilities, with given
           uniform numbers: the first drafts accepted with min(1, p / q), then
           one token of the normalised max(p - q, 0), or of p behind the last.
  fork     requests that go on from another one's tokens: full pages are
           shared (an owner more), the last one's rows are copied, in the
           caches of all layers.
  free     rows behind the ones that a request keeps: pages without another
           owner go back to the free list.
  compact  the pages in use onto the lowest numbers: tables, owners, free list,
           and the pages of all layers' caches that move.

``refs`` [pages] holds how many owners a page has beside its first.  With
``own`` false, ``run`` computes all of it by elementary torch operations; with
``own`` true, by this repository's kernels.
"""

import math

import torch

own = False

LATENT, PE, NOPE, VDIM = 512, 64, 128, 128
ROW = LATENT + PE
QK = NOPE + PE
SCALE = QK ** -0.5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the end of a chat turn behind its short history: launch latency
        dict(name="chunk_t37_h8", op="chunk", dtype="bf16", heads=8, lens_q="37", lens_k="237", page=64),
        # one step of chunked prefill: requests at different places, down to one token, small pages that end in a tile
        dict(name="chunk_mixed_h16_fp16", op="chunk", dtype="fp16", heads=16, lens_q="512,129,1,1000",
             lens_k="8192,4039,3000,1000", page=16),
        # a full batch of long prompts, eighth chunk
        dict(name="chunk_n8_t1024_h16", op="chunk", dtype="bf16", heads=16, lens_q=",".join(["1024"] * 8),
             lens_k=",".join(["8192"] * 8), page=64),
        # one conversation, four drafted tokens
        dict(name="verify_n1_s4_v32768", op="verify", dtype="fp32", requests=1, drafts=4, vocab=32768, ragged=False,
             proposer="model"),
        # drafts found in the prompt, which have no probabilities; odd vocabulary, rows at odd addresses
        dict(name="verify_n256_s5_v50257_bf16", op="verify", dtype="bf16", requests=256, drafts=5, vocab=50257,
             ragged=True, proposer="lookup"),
        # a serving batch with a draft model
        dict(name="verify_n128_s3_v131072", op="verify", dtype="fp32", requests=128, drafts=3, vocab=131072,
             ragged=False, proposer="model"),
        # eight samples of one prompt
        dict(name="fork_f8_l4", op="fork", dtype="bf16", parents=1, children=8, shortest=4039, longest=4039, page=64,
             layers=4),
        # each of many requests forked twice
        dict(name="fork_f256_l4", op="fork", dtype="bf16", parents=128, children=256, shortest=1, longest=8192, page=64,
             layers=4),
        # rejected drafts of a serving batch
        dict(name="free_n256_step", op="free", requests=256, shortest=8, longest=8192, group=1, page=16, kind="drafts"),
        # many requests end, some of whose pages others still own
        dict(name="free_n2048_ended", op="free", requests=2048, shortest=0, longest=4096, group=4, page=16, kind="ended"),
        # a small pool after a few requests have ended
        dict(name="compact_p512_l1", op="compact", dtype="fp16", requests=16, shortest=64, longest=1024, group=1, page=64,
             pages=512, layers=1),
        # a large pool, half of it in use and scattered
        dict(name="compact_p8192_l2", op="compact", dtype="bf16", requests=256, shortest=1, longest=2048, group=2, page=64,
             pages=8192, layers=2),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "verify", "fork", "free", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "chunk":
        n, heads = _between(rng, 1, 16), _between(rng, 1, 32)
        lens_q = [_between(rng, 1, 2048) for _ in range(n)]
        lens_k = [l + (0 if rng.random() < 0.2 else _between(rng, 1, 16384)) for l in lens_q]
        if n > 2 and rng.random() < 0.3:   # a request that gets nothing in this step
            lens_q[1] = 0
        while heads * n * max(max(lens_q), 1) * max(lens_k) > 1.2e9 or sum(lens_k) * heads > 1.2e6:
            lens_k = [q // 2 + (k - q) // 2 for q, k in zip(lens_q, lens_k)]
            lens_q = [q // 2 for q in lens_q]
        if sum(lens_q) == 0:
            lens_q[0], lens_k[0] = 1, lens_k[0] + 1
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), heads=heads, lens_q=",".join(map(str, lens_q)),
                    lens_k=",".join(map(str, lens_k)), page=page)
    if op == "verify":
        vocab, n, drafts = _between(rng, 100, 262144), _between(rng, 1, 512), _between(rng, 1, 15)
        while n * (drafts + 1) * vocab > 67e6:
            n, drafts = (n + 1) // 2, (drafts + 1) // 2
        return dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), requests=n, drafts=drafts, vocab=vocab,
                    ragged=rng.random() < 0.5, proposer=rng.choice(["model", "model", "lookup"]))
    longest = _between(rng, 1, 8192)
    shortest = rng.randint(0, longest)
    if op == "fork":
        children, layers = _between(rng, 1, 256), rng.randint(1, 4)
        parents = rng.randint(1, children)
        while parents * (longest // page + 1) * page * layers > 2 ** 21:
            longest, shortest = (longest + 1) // 2, shortest // 2
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), parents=parents, children=children, shortest=shortest,
                    longest=longest, page=page, layers=layers)
    requests, group = _between(rng, 1, 2048), rng.choice([1, 1, 2, 4])
    if op == "free":
        while requests * (longest // page + 1) > 2 ** 19:
            requests = requests // 2
        return dict(op=op, requests=requests, shortest=shortest, longest=longest, group=group, page=page,
                    kind=rng.choice(["drafts", "ended"]))
    layers = rng.randint(1, 2)
    while requests * (longest // page + 1) * page * layers > 2 ** 19:
        requests, longest, shortest = (requests + 1) // 2, (longest + 1) // 2, shortest // 2
    held = requests * (longest // page + 1)
    return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), requests=requests, shortest=shortest, longest=longest,
                group=group, page=page, pages=held + rng.randint(1, held + 8), layers=layers)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _spread(lo, hi, n, step=7919):
    """n lengths of [lo, hi], uneven, the longest first; the same for every seed."""
    return [hi - (i * step) % (hi - lo + 1) for i in range(n)]


def _up(a, b):
    return -(-a // b)


def _owned(lens, group, page):
    """How many of its pages a request shares with the first of its group, and how many pages that makes in all."""
    shared = [0 if i % group == 0 else min(l, lens[i - i % group]) // (2 * page) for i, l in enumerate(lens)]
    return shared, sum(_up(l, page) - s for l, s in zip(lens, shared))


def _kept(case):
    lens = _spread(case["shortest"], case["longest"], case["requests"])
    if case["kind"] == "drafts":   # up to seven rejected drafts
        return lens, [max(0, l - (i * 5) % 8) for i, l in enumerate(lens)]
    return lens, [l if i % 3 == 1 else 0 for i, l in enumerate(lens)]


def _forks(case):
    """Lengths of the parents, and each child's parent."""
    return _spread(case["shortest"], case["longest"], case["parents"]), [i % case["parents"] for i in range(case["children"])]


def work(case):
    op = case["op"]
    if op == "chunk":
        lens_q, lens_k, h = _ints(case["lens_q"]), _ints(case["lens_k"]), case["heads"]
        tq = sum(lens_q)
        tk = sum(k for q, k in zip(lens_q, lens_k) if q > 0)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(lens_q, lens_k))
        return {"bytes": tk * ROW * 2 + h * (NOPE + VDIM) * LATENT * 2 + tq * h * ((QK + VDIM) * 2 + 4)
                + sum(_up(k, case["page"]) for k in lens_k) * 4,
                "flops": 2 * tk * h * (NOPE + VDIM) * LATENT + 2 * pairs * h * (QK + VDIM)}
    if op == "verify":
        n, s, v = case["requests"], case["drafts"], case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        rows = 2 if case["proposer"] == "model" else 1   # the rows that the last token is drawn from
        return {"bytes": n * v * size * rows + n * s * (8 + 4 + size * rows) + n * ((s + 1) * 8 + 4),
                "flops": n * v * (rows + 1)}
    page = case["page"]
    if op == "fork":
        lens, parent = _forks(case)
        copies = sum(lens[p] % page != 0 for p in parent)
        full = sum(lens[p] // page for p in parent)
        rows, pages, _ = _fork_sizes(case)
        return {"bytes": copies * 2 * page * ROW * 2 * case["layers"] + full * 12 + pages * 8 + rows * 8 + copies * 16,
                "flops": full}
    lens = _spread(case["shortest"], case["longest"], case["requests"])
    held = sum(_up(l, page) for l in lens)
    used = _owned(lens, case["group"], page)[1]
    if op == "free":
        lens, keep = _kept(case)
        gone = sum(_up(l, page) - _up(k, page) for l, k in zip(lens, keep))
        return {"bytes": gone * 8 + (used + 64) * 8 + 12 * case["requests"], "flops": gone}
    moves = used * (case["pages"] - used) // case["pages"]   # of pages spread evenly
    width = max(1, max(_up(l, page) for l in lens))
    return {"bytes": moves * 2 * page * ROW * 2 * case["layers"] + case["pages"] * 24 + held * 4
            + width * case["requests"] * 4, "flops": case["pages"]}


def _fork_sizes(case):
    """Rows of the table, pages of the pool, columns of the table."""
    lens, parent = _forks(case)
    need = sum(_up(l, case["page"]) for l in lens)
    return case["parents"] + case["children"] + 3, need + len(parent) + 5, max(1, max(_up(l, case["page"]) for l in lens) + 1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(TYPES[case["dtype"]])

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    def order(pages):
        return torch.randperm(pages, generator=gen, device=dev).to(torch.int32)

    def table(need, width, pages, shared=None, group=1):
        """Tables of requests with need[i] pages, the first shared[i] of them those of its group's first request."""
        own_pages = [a - (shared[i] if shared else 0) for i, a in enumerate(need)]
        starts = ints([sum(own_pages[:i]) for i in range(len(need))], torch.int64)[:, None]
        cols = torch.arange(width, device=dev)[None, :]
        cut = ints(shared if shared else [0] * len(need), torch.int64)[:, None]
        at = starts + cols - cut
        if shared:
            at = torch.where(cols < cut, starts[torch.arange(len(need), device=dev) // group * group] + cols, at)
        cells = torch.where(cols < ints(need, torch.int64)[:, None], pages[at.clamp(0, pages.shape[0] - 1)], -1)
        return cells.to(torch.int32)

    if op == "chunk":
        lens_q, lens_k, h, page = _ints(case["lens_q"]), _ints(case["lens_k"]), case["heads"], case["page"]
        need = [_up(l, page) for l in lens_k]
        s["cache"] = normal(sum(need) + 3, page, ROW)
        s["table"] = table(need, max(1, max(need)), order(sum(need) + 3))
        s["lens"] = ints(lens_k)
        s["cu"] = ints([sum(lens_q[:i]) for i in range(len(lens_q) + 1)])
        s["q"] = normal(sum(lens_q), h, QK)
        s["w_up"] = normal(h, NOPE + VDIM, LATENT, scale=LATENT ** -0.5)
        s["keys"] = sum(lens_k)
    elif op == "verify":
        n, d, v = case["requests"], case["drafts"], case["vocab"]
        logits = torch.randn(n, d + 1, v, generator=gen, device=dev).mul_(2.5)
        s["target"] = torch.softmax(logits, -1).to(TYPES[case["dtype"]])
        if case["proposer"] == "model":   # a smaller model: the same logits, less sure of them
            draft = torch.softmax(logits[:, :d].add_(torch.randn(n, d, v, generator=gen, device=dev), alpha=0.7), -1)
            s["draft"] = draft.to(TYPES[case["dtype"]])
            pick = draft
        else:
            s["draft"], pick = None, torch.softmax(logits[:, :d] * 2, -1)
        # sampled by the largest of p / (exponential numbers)
        noise = torch.rand(n, d, v, generator=gen, device=dev).clamp_(1e-20).log_().neg_().clamp_(1e-20)
        s["tokens"] = (pick / noise).argmax(-1)
        if case["ragged"]:   # some requests have fewer drafts
            count = torch.randint(0, d + 1, (n, 1), generator=gen, device=dev)
            s["tokens"] = torch.where(torch.arange(d, device=dev) < count, s["tokens"], -1)
        s["uniform"] = torch.rand(n, d + 1, generator=gen, device=dev)
    elif op == "fork":
        lens, parent = _forks(case)
        rows, pages, width = _fork_sizes(case)
        need = [_up(l, case["page"]) for l in lens]
        pool = order(pages)
        at = order(rows)[:case["parents"] + case["children"]]   # rows that requests have
        s["table"] = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
        s["lens"] = torch.zeros(rows, dtype=torch.int32, device=dev)
        first = at[:case["parents"]].long()
        s["table"][first], s["lens"][first] = table(need, width, pool), ints(lens)
        s["parents"], s["children"] = at[ints(parent, torch.int64)], at[case["parents"]:].clone()
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["free"], s["head"] = pool, ints([sum(need)])
        s["caches"] = [normal(pages, case["page"], ROW) for _ in range(case["layers"])]
    elif op == "free":
        lens, keep = _kept(case)
        need = [_up(l, case["page"]) for l in lens]
        shared, used = _owned(lens, case["group"], case["page"])
        pool = order(used + 64)
        s["table"] = table(need, max(1, max(need)), pool, shared, case["group"])
        s["lens"], s["keep"] = ints(lens), ints(keep)
        s["refs"] = _owners(s["table"], used + 64)
        s["free"], s["head"] = pool.clone(), ints([used])
    else:
        lens = _spread(case["shortest"], case["longest"], case["requests"])
        need = [_up(l, case["page"]) for l in lens]
        shared, used = _owned(lens, case["group"], case["page"])
        pool = order(case["pages"])
        s["table"] = table(need, max(1, max(need)), pool, shared, case["group"])
        s["lens"] = ints(lens)
        s["refs"] = _owners(s["table"], case["pages"])
        s["free"], s["head"] = pool, ints([used])
        s["caches"] = [normal(case["pages"], case["page"], ROW) for _ in range(case["layers"])]
    return s


def _owners(table, pages):
    count = torch.zeros(pages + 1, dtype=torch.int32, device=table.device)
    cells = table.flatten().long()
    count.scatter_add_(0, torch.where(cells < 0, pages, cells), torch.ones_like(cells, dtype=torch.int32))
    return (count[:pages] - 1).clamp(min=0)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_chunk(s):
    q, cache, table, lens, cu, w = s["q"], s["cache"], s["table"], s["lens"], s["cu"], s["w_up"]
    n, (total, h, _) = lens.shape[0], q.shape
    lq = max(_ints(s["lens_q"]))
    at = torch.arange(lq, device=q.device)
    new = cu[1:] - cu[:-1]
    x = q[(cu[:-1, None] + at).clamp(max=total - 1)].float().transpose(1, 2)               # [N, H, lq, 192]
    rows = cache[table.clamp(min=0)].reshape(n, -1, ROW)[:, :max(_ints(s["lens_k"]))].float()
    kv = torch.einsum("njc,hdc->nhjd", rows[..., :LATENT], w.float())
    scores = x[..., :NOPE] @ kv[..., :NOPE].transpose(-1, -2)
    scores += x[..., NOPE:] @ rows[:, None, :, LATENT:].transpose(-1, -2)
    j = torch.arange(rows.shape[1], device=q.device)
    sees = (at < new[:, None])[:, :, None] & (j <= at[None, :, None] + (lens - new)[:, None, None]) & (j < lens[:, None, None])
    scores.mul_(SCALE).masked_fill_(~sees[:, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    p.masked_fill_(~sees[:, None], 0.0)
    sums = p.sum(-1, keepdim=True)
    o = (p @ kv[..., NOPE:]) / torch.where(sums > 0, sums, torch.ones_like(sums))
    lse = top + sums.log()
    tok = torch.arange(total, device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return o[seq, :, tok - cu[seq]].to(q.dtype), lse[seq, :, tok - cu[seq], 0]


def _plain_verify(s):
    tokens, target, u, draft = s["tokens"], s["target"], s["uniform"].double(), s["draft"]
    n, d = tokens.shape
    drafted = (tokens >= 0).int().cumprod(1).bool()
    at = tokens.clamp(min=0)[..., None]
    p = target[:, :d].gather(2, at)[..., 0].double()
    q = draft.gather(2, at)[..., 0].double() if draft is not None else torch.ones_like(p)
    taken = (drafted & (u[:, :d] * q < p)).int().cumprod(1).sum(1)
    rows = torch.arange(n, device=u.device)
    weight = target[rows, taken].double()
    there = (taken < drafted.sum(1))[:, None]        # a rejected draft, whose share is taken out
    turned = rows, taken.clamp(max=d - 1)
    if draft is not None:
        less = draft[turned].double()
    else:
        less = torch.zeros_like(weight).scatter_(1, at[turned], float("inf"))
    rest = torch.where(there, (weight - less).clamp(min=0), weight)
    weight = torch.where(rest.sum(1, keepdim=True) > 0, rest, weight)
    sums = weight.cumsum(1)
    last = torch.where(weight > 0, torch.arange(weight.shape[1], device=u.device), 0).amax(1)
    token = torch.minimum((sums <= u[:, d:] * sums[:, -1:]).sum(1), last)
    cols = torch.arange(d + 1, device=u.device)
    out = torch.cat([tokens, tokens.new_full((n, 1), -1)], 1)
    out = torch.where(cols < taken[:, None], out, torch.where(cols == taken[:, None], token[:, None], -1))
    return out, (taken + 1).to(torch.int32)


def _plain_copies(caches, src, dst):
    there = (src >= 0) & (dst >= 0)
    src, dst = src[there].long(), dst[there].long()
    for cache in caches:
        cache[dst] = cache[src]


def _plain_fork(s):
    table, lens, refs, free, page = s["table"], s["lens"], s["refs"], s["free"], s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    length = lens[parents]
    full, part = length // page, length % page != 0
    ends = part.cumsum(0)
    fresh = free[(s["head"] + ends - 1).clamp(0, free.shape[0] - 1)]
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    old = table[parents]
    shared = cols < full[:, None]
    table[children] = torch.where(shared, old, torch.where((cols == full[:, None]) & part[:, None], fresh[:, None],
                                                           table[children]))
    more = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=refs.device)
    more.scatter_add_(0, torch.where(shared, old, refs.shape[0]).flatten().long(), shared.flatten().int())
    src = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0]
    pairs = torch.where(part[:, None], torch.stack([src, fresh], 1), -1)
    _plain_copies(s["caches"], pairs[:, 0], pairs[:, 1])
    return lens.index_copy(0, children, length), refs + more[:-1], s["head"] + ends[-1:].to(torch.int32), pairs, table, s["caches"]


def _plain_free(s):
    table, lens, keep, refs, free, page = s["table"], s["lens"], s["keep"], s["refs"], s["free"], s["page"]
    pages = refs.shape[0]
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    gone = (cols >= ((keep + page - 1) // page)[:, None]) & (cols < ((lens + page - 1) // page)[:, None])
    count = torch.zeros(pages + 1, dtype=torch.int32, device=refs.device)
    count.scatter_add_(0, torch.where(gone, table, pages).flatten().long(), gone.flatten().int())
    freed = count[:pages] > refs
    ends = freed.cumsum(0)
    head = s["head"] - ends[-1:].to(torch.int32)
    at = torch.arange(pages, device=refs.device)[freed]
    free[(head + ends - 1)[freed]] = at.to(torch.int32)
    return keep.clone(), (refs - count[:pages]).clamp(min=0), head, free


def _plain_compact(s):
    table, lens, refs, free, page = s["table"], s["lens"], s["refs"], s["free"], s["page"]
    pages, dev = refs.shape[0], table.device
    listed_free = torch.arange(free.shape[0], device=dev) >= s["head"]
    is_free = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    is_free[torch.where(listed_free, free, pages).long()] = True
    is_free = is_free[:pages]
    at = torch.arange(pages, device=dev)
    used = pages - is_free.sum()
    before = is_free.cumsum(0) - is_free.int()
    hole, mover = is_free & (at < used), ~is_free & (at >= used)
    holes = hole.sum()
    rank = torch.where(hole, before, (at - used) - (before - holes))
    pairs = torch.full((pages // 2, 2), -1, dtype=torch.int32, device=dev)
    pairs[rank[mover], 0] = at[mover].int()
    pairs[rank[hole], 1] = at[hole].int()
    moved = torch.where(is_free, -1, at).int()
    moved[at[mover]] = pairs[rank[mover], 1]
    refs_out = torch.zeros_like(refs)
    refs_out[moved[~is_free].long()] = refs[~is_free]
    cols = torch.arange(table.shape[1], device=dev)[None, :]
    held = cols < ((lens + page - 1) // page)[:, None]
    table_out = torch.where(held, moved[table.clamp(min=0).long()], -1)
    place = torch.arange(free.shape[0], device=dev) - s["head"]
    free_out = torch.where(listed_free, used + place, free).int()
    _plain_copies(s["caches"], pairs[:, 0], pairs[:, 1])
    return table_out, refs_out, free_out, pairs, holes.int().reshape(1), moved, s["caches"]


def run(state):
    s, op = state, state["op"]
    if own:
        from chunked_gated_delta_kda_gb300 import drafts, latent, pages
        if op == "chunk":
            return latent.latent_chunk(s["q"], s["cache"], s["table"], s["lens"], s["w_up"], s["cu"], s["keys"])
        if op == "verify":
            return drafts.verify_drafts(s["tokens"], s["target"], s["uniform"], draft_probs=s["draft"])
        if op == "fork":
            lens, refs, head, pairs = pages.page_fork(s["table"], s["lens"], s["parents"], s["children"], s["refs"],
                                                      s["free"], s["head"], s["page"])
            return lens, refs, head, pairs, s["table"], pages.page_copy(s["caches"], pairs)
        if op == "free":
            return pages.page_free(s["table"], s["lens"], s["keep"], s["refs"], s["free"], s["head"], s["page"]) + (s["free"],)
        table, refs, free, pairs, count, moved = pages.page_compact(s["table"], s["lens"], s["refs"], s["free"], s["head"],
                                                                    s["page"])
        return table, refs, free, pairs, count, moved, pages.page_copy(s["caches"], pairs, count=count)
    return {"chunk": _plain_chunk, "verify": _plain_verify, "fork": _plain_fork, "free": _plain_free,
            "compact": _plain_compact}[op](s)


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence and head at a time.  The other
# operators' outputs are whole numbers and copies.
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "chunk":
        return None
    s = prepare(case, seed)
    total, h, _ = s["q"].shape
    o = torch.zeros(total, h, VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full((total, h), -float("inf"), dtype=torch.float64, device="cuda")
    a = 0
    for i, (lq, lk) in enumerate(zip(_ints(case["lens_q"]), _ints(case["lens_k"]))):
        if lq == 0:
            continue
        own_pages = s["table"][i, :_up(lk, case["page"])].long()
        rows = s["cache"][own_pages].reshape(-1, ROW)[:lk].double()
        hidden = torch.ones(lq, lk, dtype=torch.bool, device="cuda").triu(lk - lq + 1)
        for j in range(h):
            up = s["w_up"][j].double()
            k = torch.cat([rows[:, :LATENT] @ up[:NOPE].T, rows[:, LATENT:]], 1)
            x = (s["q"][a:a + lq, j].double() @ k.T * SCALE).masked_fill_(hidden, -float("inf"))
            lse[a:a + lq, j] = torch.logsumexp(x, 1)
            o[a:a + lq, j] = torch.softmax(x, 1) @ (rows[:, :LATENT] @ up[NOPE:].T)
        a += lq
    return o, lse
