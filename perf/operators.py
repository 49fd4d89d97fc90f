"""Latent attention and its paged cache: the cases that are measured, and the operators' plain forms.

Latent attention keeps one shared row a token, 512 latent channels and 64
positional ones, from which every head's key and value come.  Five operators:

  prefill  expanded form, forward: queries [T, H, 128 + 64], keys and values
           expanded to [T, H, 128 + 128], the positional key [T, 64] shared by
           the heads; output [T, H, 128] and the rows' log-sum-exp.
  train    its backward: the gradients of the queries, of the expanded keys
           and values, and of the shared positional key (summed over heads).
  decode   absorbed form over the paged cache: queries [N, S, H, 512 + 64]
           against the cached rows, values are their first 512 channels.
  append   new tokens' latent rows, RMS-normalised, into their cache slots.
  tables   block tables and slot maps from the requests' lengths.

With ``own`` false, ``run`` computes them by elementary torch operations in
32 bits; with ``own`` true, by this repository's kernels.
"""

import torch

own = False

LATENT, PE, NOPE, VDIM = 512, 64, 128, 128
ROW = LATENT + PE
QK = NOPE + PE
SCALE = QK ** -0.5
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short prompt: launch latency and a tile that is mostly empty
        dict(name="prefill_t37_h32", op="prefill", dtype="bf16", heads=32, lens_q="37", lens_k="37", causal=True),
        # chunked prefill: new tokens of several requests behind prefixes that are already cached, down to one token
        dict(name="prefill_chunks_h16_fp16", op="prefill", dtype="fp16", heads=16, lens_q="512,129,1,1000",
             lens_k="8192,4039,3000,1000", causal=True),
        # long prompts of equal length
        dict(name="prefill_b4_t8192_h16", op="prefill", dtype="bf16", heads=16, lens_q="8192,8192,8192,8192",
             lens_k="8192,8192,8192,8192", causal=True),
        # training on two short sequences
        dict(name="train_b2_t2048_h8", op="train", dtype="bf16", heads=8, lens_q="2048,2048", lens_k="2048,2048",
             causal=True),
        # training on a packed batch of documents of uneven lengths
        dict(name="train_varlen6_t9192_h32", op="train", dtype="bf16", heads=32, lens_q="400,624,1000,3000,129,4039",
             lens_k="400,624,1000,3000,129,4039", causal=True),
        # one long conversation, one token a step: the cache axis has to be split over the whole GPU
        dict(name="decode_n1_h32_l65536", op="decode", dtype="bf16", requests=1, tokens=1, heads=32, shortest=65536,
             longest=65536, page=64),
        # a full serving batch of uneven lengths
        dict(name="decode_n256_h32_l8192", op="decode", dtype="bf16", requests=256, tokens=1, heads=32, shortest=1,
             longest=8192, page=64),
        # speculative decoding: four tokens a request to verify, small pages that end inside a tile
        dict(name="decode_n64_s4_h16_fp16", op="decode", dtype="fp16", requests=64, tokens=4, heads=16, shortest=100,
             longest=4039, page=16),
        # the cache rows of one decode step
        dict(name="append_n256", op="append", dtype="bf16", tokens=256, page=64, pages=4096, norm=True),
        # the cache rows of a packed prefill
        dict(name="append_t9192", op="append", dtype="bf16", tokens=9192, page=64, pages=4096, norm=True),
        # tables and slots of a decode step: one new token a request
        dict(name="tables_n256_step", op="tables", requests=256, shortest=1, longest=8192, new_shortest=1,
             new_longest=1, page=64, width=256),
        # tables and slots of a large mixed step: new tokens from none to long prompts
        dict(name="tables_n2048_prefill", op="tables", requests=2048, shortest=0, longest=4096, new_shortest=0,
             new_longest=512, page=16, width=512),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "train", "decode", "append", "tables"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("prefill", "train"):
        n, heads, causal = _between(rng, 1, 8), _between(rng, 1, 32), rng.random() < 0.8
        lens_q = [_between(rng, 1, 4096) for _ in range(n)]
        kind = rng.random()   # equal lengths, a prefix before the queries, or lengths of their own
        lens_k = [l if kind < 0.5 else l + _between(rng, 1, 4096) if kind < 0.9 else _between(rng, 1, 4096)
                  for l in lens_q]
        while n * heads * max(lens_q) * max(lens_k) > 1.2e9:
            lens_q = [max(1, l // 2) for l in lens_q]
            lens_k = [max(1, l // 2) for l in lens_k]
        return dict(op=op, dtype=dtype, heads=heads, lens_q=",".join(map(str, lens_q)),
                    lens_k=",".join(map(str, lens_k)), causal=causal)
    if op == "decode":
        n, s, heads = _between(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 7]), _between(rng, 1, 128)
        longest = _between(rng, 1, 65536)
        while n * longest > 2 ** 20 or n * s * heads * longest > 2 ** 25:
            longest, s = max(1, longest // 2), (s + 1) // 2
        return dict(op=op, dtype=dtype, requests=n, tokens=s, heads=heads, shortest=rng.randint(0, longest),
                    longest=longest, page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        t, page = _between(rng, 1, 16384), rng.choice([16, 32, 64, 128])
        return dict(op=op, dtype=dtype, tokens=t, page=page, pages=-(-t // page) + rng.randint(1, 500),
                    norm=rng.random() < 0.7)
    n, page = _between(rng, 1, 2048), rng.choice([16, 32, 64, 128])
    longest, new_longest = _between(rng, 1, 4096), _between(rng, 1, 512)
    return dict(op=op, requests=n, shortest=rng.randint(0, longest), longest=longest,
                new_shortest=rng.randint(0, new_longest), new_longest=new_longest, page=page,
                width=-(-(longest + new_longest) // page) + rng.randint(0, 3))


def _lens(text):
    return [int(x) for x in text.split(",")]


def _spread(lo, hi, n, step=7919):
    """n lengths of [lo, hi], uneven, the longest first; the same for every seed."""
    return [hi - (i * step) % (hi - lo + 1) for i in range(n)]


def _equal(case):
    q, k = _lens(case["lens_q"]), _lens(case["lens_k"])
    return len(set(q)) == 1 and q == k


def _pairs(case):
    """Query-key pairs that the mask leaves, a head."""
    total = 0
    for lq, lk in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
        if not case["causal"]:
            total += lq * lk
        else:   # query i sees keys up to i + lk - lq
            first = max(0, lq - lk)          # the first query that sees any
            n = lq - first
            total += n * (lk - lq + first + 1) + n * (n - 1) // 2 if n > 0 else 0
    return total


def work(case):
    op = case["op"]
    if op in ("prefill", "train"):
        tq, tk, h = sum(_lens(case["lens_q"])), sum(_lens(case["lens_k"])), case["heads"]
        read = tq * h * QK * 2 + tk * h * (NOPE + VDIM) * 2 + tk * PE * 2
        if op == "prefill":
            return {"bytes": read + tq * h * (VDIM * 2 + 4), "flops": 2 * _pairs(case) * h * (QK + VDIM)}
        grads = read
        return {"bytes": read + tq * h * (2 * VDIM * 2 + 4) + grads, "flops": 2 * _pairs(case) * h * (3 * QK + 2 * VDIM)}
    if op == "decode":
        n, s, h = case["requests"], case["tokens"], case["heads"]
        lens = _spread(case["shortest"], case["longest"], n)
        pairs = sum(max(0, l - s + 1 + t) for l in lens for t in range(s))
        return {"bytes": sum(lens) * ROW * 2 + n * s * h * ((ROW + LATENT) * 2 + 4) + sum(-(-l // case["page"]) for l in lens) * 4 + 4 * n,
                "flops": 2 * pairs * h * (ROW + LATENT)}
    if op == "append":
        return {"bytes": case["tokens"] * (2 * ROW * 2 + 8) + (LATENT * 2 if case["norm"] else 0),
                "flops": case["tokens"] * LATENT * 4 if case["norm"] else 0}
    lens, new = _spread(case["shortest"], case["longest"], case["requests"]), _new(case)
    page = case["page"]
    pages = sum(-(-(a + b) // page) + -(-a // page) * -1 for a, b in zip(lens, new))
    return {"bytes": case["requests"] * 16 + sum(new) * 8 + pages * 8, "flops": sum(new) * 4}


def _new(case):
    return _spread(case["new_shortest"], case["new_longest"], case["requests"], step=104729)


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

    if op in ("prefill", "train"):
        lens_q, lens_k, h = _lens(case["lens_q"]), _lens(case["lens_k"]), case["heads"]
        if _equal(case):   # equal lengths: no packing
            lead_q = lead_k = (len(lens_q), lens_q[0])
            s["cu_q"] = s["cu_k"] = None
        else:
            lead_q, lead_k = (1, sum(lens_q)), (1, sum(lens_k))
            s["cu_q"] = ints([sum(lens_q[:i]) for i in range(len(lens_q) + 1)])
            s["cu_k"] = ints([sum(lens_k[:i]) for i in range(len(lens_k) + 1)])
        s["q"] = normal(*lead_q, h, QK)
        s["kv"] = normal(*lead_k, h, NOPE + VDIM)
        s["k_pe"] = normal(*lead_k, ROW)[..., LATENT:]   # a slice of the latent projection's rows, as the model has it
        if op == "train":
            s["do"] = normal(*lead_q, h, VDIM)
            s["o"], s["lse"] = _plain_prefill(s)
    elif op == "decode":
        n, page = case["requests"], case["page"]
        lens = _spread(case["shortest"], case["longest"], n)
        need = [-(-l // page) for l in lens]
        total, width = sum(need) + 3, max(1, max(need))
        s["cache"] = normal(total, page, ROW)
        order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
        cols = torch.arange(width, device=dev)[None, :]
        starts = ints([sum(need[:i]) for i in range(n)], torch.int64)[:, None]
        used = cols < ints(need, torch.int64)[:, None]
        s["table"] = torch.where(used, order[(starts + cols).clamp(max=total - 1)], -1).to(torch.int32)
        s["lens"] = ints(lens)
        s["q"] = normal(n, case["tokens"], case["heads"], ROW)
    elif op == "append":
        rows, slots = case["tokens"], case["pages"] * case["page"]
        s["cache"] = normal(case["pages"], case["page"], ROW)
        s["rows"] = normal(rows, ROW, scale=3.0)
        s["slots"] = torch.randperm(slots, generator=gen, device=dev)[:rows]
        # padded entries of a captured step
        s["slots"] = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.02, -1, s["slots"])
        s["weight"] = (1 + 0.1 * torch.randn(LATENT, generator=gen, device=dev)).to(TYPES[case["dtype"]]) if case["norm"] else None
    else:
        n, page, width = case["requests"], case["page"], case["width"]
        lens, new = _spread(case["shortest"], case["longest"], n), _new(case)
        held = [-(-l // page) for l in lens]
        taken = sum(-(-(a + b) // page) for a, b in zip(lens, new)) - sum(held)
        pages = sum(held) + taken + 64
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        cols = torch.arange(width, device=dev)[None, :]
        starts = ints([sum(held[:i]) for i in range(n)], torch.int64)[:, None]
        used = cols < ints(held, torch.int64)[:, None]
        s["table"] = torch.where(used, order[(starts + cols).clamp(max=pages - 1)], -1).to(torch.int32)
        s["free"] = order[sum(held):].clone()
        s["head"] = ints([7])
        s["lens"], s["new"], s["total"] = ints(lens), ints(new), sum(new)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rows(x, cu, longest):
    """Packed rows [1, T, ...] as [N, longest, ...] in 32 bits, and which of them are there."""
    if cu is None:
        return x.float(), torch.ones(x.shape[:2], dtype=torch.bool, device=x.device)
    at = torch.arange(longest, device=x.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    return x[0][(cu[:-1, None] + at).clamp(max=x.shape[1] - 1)].float(), there


def _packed(x, like, cu):
    """The rows of _rows back in their packing."""
    if cu is None:
        return x.to(like.dtype)
    total = like.shape[1]
    at = torch.arange(total, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return x[seq, at - cu[seq]][None].to(like.dtype)


def _scores(s):
    """Masked scores [N, H, Lq, Lk], and the padded operands."""
    lq, lk = max(_lens(s["lens_q"])), max(_lens(s["lens_k"]))
    q, there_q = _rows(s["q"], s["cu_q"], lq)
    kv, there_k = _rows(s["kv"], s["cu_k"], lk)
    pe, _ = _rows(s["k_pe"], s["cu_k"], lk)
    q, kv = q.transpose(1, 2), kv.transpose(1, 2)
    k, v = torch.cat([kv[..., :NOPE], pe[:, None].expand(-1, kv.shape[1], -1, -1)], -1), kv[..., NOPE:]
    sees = (there_q[:, :, None] & there_k[:, None, :])
    if s["causal"]:
        nq, nk = there_q.sum(1), there_k.sum(1)
        i, j = torch.arange(lq, device=q.device), torch.arange(lk, device=q.device)
        sees &= j[None, None, :] <= i[None, :, None] + (nk - nq)[:, None, None]
    x = (q @ k.transpose(-1, -2)).mul_(SCALE).masked_fill_(~sees[:, None], float("-inf"))
    return x, q, k, v


def _plain_prefill(s):
    x, q, k, v = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    o = _packed(o.transpose(1, 2), s["q"], s["cu_q"])
    lse = lse.transpose(1, 2)
    return o, (lse if s["cu_q"] is None else _packed(lse, lse.new_empty(1, s["q"].shape[1], 1), s["cu_q"])).contiguous()


def _plain_train(s):
    x, q, k, v = _scores(s)
    do, _ = _rows(s["do"], s["cu_q"], q.shape[2])
    o, _ = _rows(s["o"], s["cu_q"], q.shape[2])
    lse, _ = _rows(s["lse"], s["cu_q"], q.shape[2])
    do, o, lse = do.transpose(1, 2), o.transpose(1, 2), lse.transpose(1, 2)[..., None]
    p = x.sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).exp_()
    dv = p.transpose(-1, -2) @ do
    dx = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    dq, dk = dx @ k, dx.transpose(-1, -2) @ q
    dkv = torch.cat([dk[..., :NOPE], dv], -1).transpose(1, 2)
    return (_packed(dq.transpose(1, 2), s["q"], s["cu_q"]), _packed(dkv, s["kv"], s["cu_k"]),
            _packed(dk[..., NOPE:].sum(1), s["k_pe"], s["cu_k"]))


def _plain_decode(s):
    q, cache, table, lens = s["q"], s["cache"], s["table"], s["lens"]
    n, t, h, _ = q.shape
    rows = cache[table.clamp(min=0)].reshape(n, -1, ROW).float()
    x = (q.float().reshape(n, t * h, ROW) @ rows.transpose(-1, -2)).mul_(SCALE).reshape(n, t, h, -1)
    at = torch.arange(rows.shape[1], device=q.device)
    sees = at < (lens[:, None] - t + 1 + torch.arange(t, device=q.device))[:, :, None]
    x.masked_fill_(~sees[:, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(n, t * h, -1) @ rows[..., :LATENT]).reshape(n, t, h, LATENT)
    return (o / torch.where(total > 0, total, torch.ones_like(total))).to(q.dtype), (top + total.log())[..., 0]


def _plain_append(s):
    x, cache = s["rows"].float(), s["cache"]
    c, pe = x[:, :LATENT], x[:, LATENT:]
    if s["norm"]:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    there = s["slots"] >= 0
    cache.view(-1, ROW)[s["slots"][there]] = torch.cat([c, pe], -1).to(cache.dtype)[there]
    return cache


def _plain_tables(s):
    lens, new, table, free, page = s["lens"], s["new"], s["table"], s["free"], s["page"]
    after = lens + new
    held, want = (lens + page - 1) // page, (after + page - 1) // page
    take = want - held
    ends = take.cumsum(0)
    head = s["head"] + ends[-1:].to(torch.int32)
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    at = s["head"] + (ends - take)[:, None] + cols - held[:, None]
    fresh = (cols >= held[:, None]) & (cols < want[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, free.shape[0] - 1)], table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
    tok = torch.arange(s["total"], device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = lens[seq] + tok - cu[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    return slots, cu, after, head, table


def run(state):
    s, op = state, state["op"]
    if own:
        from chunked_gated_delta_kda_gb300 import latent
        if op == "prefill":
            return latent.latent_fwd(s["q"], s["kv"], s["k_pe"], causal=s["causal"], cu_seqlens_q=s["cu_q"],
                                     cu_seqlens_k=s["cu_k"])
        if op == "train":
            return latent.latent_bwd(s["q"], s["kv"], s["k_pe"], s["o"], s["lse"], s["do"], causal=s["causal"],
                                     cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"])
        if op == "decode":
            return latent.latent_decode(s["q"], s["cache"], s["table"], s["lens"])
        if op == "append":
            return latent.latent_append(s["rows"], s["slots"], s["cache"], norm_weight=s["weight"], eps=EPS)
        return latent.block_tables(s["lens"], s["new"], s["table"], s["free"], s["head"], s["page"], s["total"]) + (s["table"],)
    return {"prefill": _plain_prefill, "train": _plain_train, "decode": _plain_decode, "append": _plain_append,
            "tables": _plain_tables}[op](s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "append":
        out = s["cache"].double()
        x = s["rows"].double()
        if case["norm"]:
            x[:, :LATENT] *= ((x[:, :LATENT] ** 2).sum(-1, keepdim=True) / LATENT + EPS) ** -0.5
            x[:, :LATENT] *= s["weight"].double()
        flat = out.view(-1, ROW)
        for slot, row in zip(s["slots"].tolist(), x):
            if slot >= 0:
                flat[slot] = row
        return out
    if op == "decode":
        n, t, h, _ = s["q"].shape
        o, lse = torch.zeros(n, t, h, LATENT, dtype=torch.float64, device="cuda"), torch.full((n, t, h), -float("inf"), dtype=torch.float64, device="cuda")
        for i, l in enumerate(s["lens"].tolist()):
            pages = s["table"][i, :-(-l // case["page"])].long()
            rows = s["cache"][pages].reshape(-1, ROW)[:l].double()
            for j in range(t):
                seen = l - t + 1 + j
                if seen > 0:
                    x = s["q"][i, j].double() @ rows[:seen].T * SCALE
                    lse[i, j] = torch.logsumexp(x, -1)
                    o[i, j] = torch.softmax(x, -1) @ rows[:seen, :LATENT]
        return o, lse
    h, flat = case["heads"], lambda x: x.reshape(-1, *x.shape[2:])
    q, kv, pe = flat(s["q"]), flat(s["kv"]), flat(s["k_pe"])
    o = torch.zeros(*q.shape[:2], VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64, device="cuda")
    dq, dkv, dpe = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, kv, pe))
    a = b = 0
    for lq, lk in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
        for i in range(h):
            qi, vi = q[a:a + lq, i].double(), kv[b:b + lk, i, NOPE:].double()
            ki = torch.cat([kv[b:b + lk, i, :NOPE].double(), pe[b:b + lk].double()], -1)
            x = qi @ ki.T * SCALE
            if case["causal"]:
                x.masked_fill_(torch.ones(lq, lk, dtype=torch.bool, device="cuda").triu(lk - lq + 1), -float("inf"))
            li = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(li), torch.zeros_like(li), li)[:, None])
            lse[a:a + lq, i], o[a:a + lq, i] = li, p @ vi
            if op == "train":
                di = flat(s["do"])[a:a + lq, i].double()
                dx = p * (di @ vi.T - (di * o[a:a + lq, i]).sum(-1, keepdim=True)) * SCALE
                dq[a:a + lq, i] = dx @ ki
                dk = dx.T @ qi
                dkv[b:b + lk, i, :NOPE], dkv[b:b + lk, i, NOPE:] = dk[:, :NOPE], p.T @ di
                dpe[b:b + lk] += dk[:, NOPE:]
        a, b = a + lq, b + lk
    if op == "prefill":
        return o.reshape(*s["q"].shape[:3], VDIM), lse.reshape(s["q"].shape[:3])
    return dq.reshape(s["q"].shape), dkv.reshape(s["kv"].shape), dpe.reshape(s["k_pe"].shape)
