"""A latent-attention layer served and trained: the latent operators together.

``LatentLayer`` holds random weights of one layer of H heads over a hidden
size D (the projections are plain matrix products) and runs

* ``prefill``: block tables for the prompts, their rows into the paged cache,
  attention in the expanded form,
* ``chunk``: the same for new tokens of requests that have cached ones, over
  the paged cache,
* ``decode``: one token a request: tables, cache row, attention in the
  absorbed form, whose query takes the key projection and whose output the
  value projection,
* ``fork``, ``keep``, ``compact``: requests that go on from another one's
  tokens, end or lose their last ones, and the pages in use onto the lowest
  numbers,
* ``train``: forward and backward in the expanded form, with the gradient of
  the layer's input.

``Decoder`` puts such a layer between an embedding and an output projection
and draws tokens, several a step where drafts of them are at hand.

``python -m chunked_gated_delta_kda_gb300.latent_serving`` prefills a ragged
batch, decodes a few tokens and compares every decoded token's output with the
expanded form over its whole sequence; then it lets a decoder continue forked
requests with drafts found in their own tokens.
"""

from __future__ import annotations

import torch

from . import binding, drafts, latent, pages
from .latent import KEY_CHANNELS, LATENT_CHANNELS, PE_CHANNELS, ROW_CHANNELS, VALUE_CHANNELS


class LatentLayer:
    def __init__(self, hidden: int, heads: int, requests: int, pages: int, page_size: int = 64, width: int = 64,
                 dtype=torch.bfloat16, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5).to(dtype)

        self.heads = heads
        self.w_q = weight(heads * (KEY_CHANNELS + PE_CHANNELS), hidden)
        self.w_row = weight(ROW_CHANNELS, hidden)                       # latent and positional channels of a token
        self.norm = torch.ones(LATENT_CHANNELS, dtype=dtype, device=device)
        self.w_up = weight(heads, KEY_CHANNELS + VALUE_CHANNELS, LATENT_CHANNELS)
        i32 = dict(dtype=torch.int32, device=device)
        self.cache = torch.zeros(pages, page_size, ROW_CHANNELS, dtype=dtype, device=device)
        self.page_size = page_size
        self.table = torch.full((requests, width), -1, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.free = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
        self.head = torch.zeros(1, **i32)
        self.refs = torch.zeros(pages, **i32)                           # owners of a page beside its first
        self.status = torch.zeros(latent.STATUS_BYTES, dtype=torch.uint8, device=device)

    def _query(self, x):
        return (x @ self.w_q.T).view(*x.shape[:-1], self.heads, KEY_CHANNELS + PE_CHANNELS)

    def _advance(self, rows, new_lens):
        """Pages for new_lens [N] tokens, and their rows [T, 576] (latent channels normalised) into the cache.  Where
        a token gets no page (slot -1, which must not be looked up) or there is not one row a token, raises and leaves
        lengths and cache as they were."""
        slots, cu, lens, head = latent.block_tables(self.lens, new_lens, self.table, self.free, self.head, self.page_size,
                                                    rows.shape[0], workspace=self.status)
        status = binding.get_status(self.status)
        if status != 0:
            raise binding.KdaError(status, "LatentLayer")
        if int(cu[-1]) != rows.shape[0]:
            raise ValueError(f"{rows.shape[0]} rows for {int(cu[-1])} new tokens")
        self.lens, self.head = lens, head
        latent.latent_append(rows, slots, self.cache, norm_weight=self.norm)
        return slots, cu

    def _expand(self, rows):
        """Keys and values of normalised rows [..., 576]: [..., H, 256]."""
        return torch.einsum("...c,hdc->...hd", rows[..., :LATENT_CHANNELS], self.w_up)

    def prefill(self, x, new_lens):
        """Packed prompts x [T, D], new_lens int32 [N], of requests that have nothing cached (0 tokens go to the
        others).  Returns [T, H, 128]."""
        if bool(((self.lens > 0) & (new_lens > 0)).any()):
            raise ValueError("prefill sees the new tokens alone: a request with cached ones goes on with chunk or decode")
        slots, cu = self._advance(x @ self.w_row.T, new_lens)
        rows = self.cache.view(-1, ROW_CHANNELS)[slots]                 # as the cache holds them
        o, _ = latent.latent_fwd(self._query(x)[None], self._expand(rows)[None], rows[None, :, LATENT_CHANNELS:],
                                 cu_seqlens_q=cu, cu_seqlens_k=cu)
        return o[0]

    def chunk(self, x, new_lens):
        """Packed new tokens x [T, D], new_lens int32 [N], of requests with or without cached ones.  Returns
        [T, H, 128]."""
        _, cu = self._advance(x @ self.w_row.T, new_lens)
        keys = int(torch.where(new_lens > 0, self.lens, 0).sum())
        o, _ = latent.latent_chunk(self._query(x), self.cache, self.table, self.lens, self.w_up, cu, keys, workspace=self.status)
        self._check()
        return o

    def _check(self):
        status = binding.get_status(self.status)
        if status != 0:
            raise binding.KdaError(status, "LatentLayer")

    def fork(self, parents, children, lens=None):
        """Requests children (int32 [F], with nothing cached) go on from the tokens of requests parents (int32 [F]), all
        of them or the first lens (int32 [F])."""
        lens_out, refs, head, pairs = pages.page_fork(self.table, self.lens, parents, children, self.refs, self.free, self.head,
                                                  self.page_size, fork_lens=lens, workspace=self.status)
        self._check()
        self.lens, self.refs, self.head = lens_out, refs, head
        pages.page_copy(self.cache, pairs)

    def keep(self, lens):
        """Each request keeps its first lens (int32 [N]) tokens, none where it ends; pages go back to the free list."""
        lens, refs, head = pages.page_free(self.table, self.lens, lens, self.refs, self.free, self.head, self.page_size,
                                           workspace=self.status)
        self._check()
        self.lens, self.refs, self.head = lens, refs, head

    def compact(self):
        """The pages in use onto the lowest numbers.  Returns how many moved."""
        table, refs, free, pairs, count, _ = pages.page_compact(self.table, self.lens, self.refs, self.free, self.head,
                                                                self.page_size, workspace=self.status)
        self._check()
        pages.page_copy(self.cache, pairs, count=count)
        self.table, self.refs, self.free = table, refs, free
        return int(count)

    def decode(self, x):
        """One token a request, x [N, D].  Returns [N, H, 128]."""
        self._advance(x @ self.w_row.T, torch.ones_like(self.lens))
        q = self._query(x)
        w_key, w_value = self.w_up[:, :KEY_CHANNELS], self.w_up[:, KEY_CHANNELS:]
        absorbed = torch.cat([torch.einsum("nhd,hdc->nhc", q[..., :KEY_CHANNELS], w_key), q[..., KEY_CHANNELS:]], -1)
        o, _ = latent.latent_decode(absorbed[:, None], self.cache, self.table, self.lens)
        return torch.einsum("nhc,hdc->nhd", o[:, 0], w_value)

    def train(self, x, grad):
        """x [B, T, D] through the expanded form (rows as they are, without the norm), grad [B, T, H, 128] on its
        output.  Returns (output, gradient of x)."""
        q, rows = self._query(x), x @ self.w_row.T
        kv, k_pe = self._expand(rows), rows[..., LATENT_CHANNELS:]
        o, lse = latent.latent_fwd(q, kv, k_pe)
        dq, dkv, dk_pe = latent.latent_bwd(q, kv, k_pe, o, lse, grad)
        drow = torch.cat([torch.einsum("bthd,hdc->btc", dkv, self.w_up), dk_pe], -1)
        return o, dq.flatten(2) @ self.w_q + drow @ self.w_row


class Decoder:
    """A latent layer between an embedding and an output projection, both random, and `temper` times its logits."""

    def __init__(self, vocab: int, hidden: int, heads: int, requests: int, pages: int, temper: float = 4.0, seed: int = 0, **layer):
        self.layer = LatentLayer(hidden, heads, requests, pages, seed=seed, **layer)
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.embed, self.out = r(vocab, hidden).to(torch.bfloat16), r(vocab, heads * VALUE_CHANNELS)
        self.temper = temper

    def probabilities(self, tokens, new_lens):
        """Of the tokens behind each of the packed tokens [T] (int64) that the requests get: fp32 [T, V]."""
        o = self.layer.chunk(self.embed[tokens], new_lens).flatten(1).float()
        o = o / o.norm(dim=1, keepdim=True)
        return torch.softmax(self.temper * (o @ self.out.T), -1)

    def start(self, prompts, new_lens, uniform):
        """Prompts (packed, int64) and a number of [0, 1) a request: the first token behind each, [N]."""
        p = self.probabilities(prompts, new_lens)[new_lens.cumsum(0) - 1]
        return drafts.verify_drafts(prompts.new_empty(len(new_lens), 0), p[:, None], uniform[:, None])[0][:, 0]

    def step(self, last, drafted, uniform, proposed=None):
        """The last token of each request [N], S drafted ones behind it [N, S] (proposed [N, S, V]: the probabilities
        that they were drawn from, if any), uniform [N, S + 1].  Returns (tokens [N, S + 1], num_accepted [N]) as
        ``drafts.verify_drafts``; the cache keeps the rows of the tokens before the last one of those."""
        n, s = drafted.shape
        p = self.probabilities(torch.cat([last[:, None], drafted.clamp(min=0)], 1).flatten(),
                               torch.full((n,), s + 1, dtype=torch.int32, device=last.device)).view(n, s + 1, -1)
        tokens, accepted = drafts.verify_drafts(drafted, p, uniform, draft_probs=proposed)
        self.layer.keep(self.layer.lens - (s + 1) + accepted)
        return tokens, accepted


def continue_forked(copies: int = 3, steps: int = 12, look: int = 3, seed: int = 3) -> float:
    """A prompt is read once and continued by `copies` requests, each with drafts found behind the last place where its
    last token stood.  Returns the tokens a step and request."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dec = Decoder(40, 256, 4, copies, pages=64, width=16, page_size=16, temper=12.0, seed=seed)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    prompt = torch.randint(0, 40, (100,), generator=gen, device="cuda")
    dec.probabilities(prompt[:-1], i32(99, *[0] * (copies - 1)))
    dec.layer.fork(i32(*[0] * (copies - 1)), i32(*range(1, copies)))
    texts = [prompt.tolist() for _ in range(copies)]
    for _ in range(steps):
        found = []
        for text in texts:
            at = next((i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]), None)
            found.append((text[at + 1:at + 1 + look] if at is not None else []) + [-1] * look)
        drafted = torch.tensor([f[:look] for f in found], device="cuda")
        last = torch.tensor([text[-1] for text in texts], device="cuda")
        tokens, accepted = dec.step(last, drafted, torch.rand(copies, look + 1, generator=gen, device="cuda"))
        for text, row, count in zip(texts, tokens.tolist(), accepted.tolist()):
            text += row[:count]
    dec.layer.keep(torch.where(torch.arange(copies, device="cuda") > 0, dec.layer.lens, 0).to(torch.int32))
    moved = dec.layer.compact()
    rate = sum(len(text) - 100 for text in texts) / (steps * copies)
    print(f"{copies} requests from one prompt of 100 tokens, {steps} steps with up to {look} drafts: {rate:.2f} tokens a step; "
          f"{moved} pages moved after the first had ended")
    return rate


def main() -> float:
    """Largest relative difference between a decoded token's output and the expanded form's."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens, steps, hidden = [400, 1, 129, 64], 3, 512
    layer = LatentLayer(hidden, 8, len(lens), pages=32, width=8)
    prompts = [torch.randn(n, hidden, generator=gen, device="cuda").to(torch.bfloat16) for n in lens]
    layer.prefill(torch.cat(prompts), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    worst = 0.0
    for _ in range(steps):
        x = torch.randn(len(lens), hidden, generator=gen, device="cuda").to(torch.bfloat16)
        prompts = [torch.cat([p, t[None]]) for p, t in zip(prompts, x)]
        out = layer.decode(x)
        fresh = LatentLayer(hidden, 8, len(lens), pages=32, width=8)
        whole = fresh.prefill(torch.cat(prompts), torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda"))
        last = torch.tensor([len(p) for p in prompts], device="cuda").cumsum(0) - 1
        worst = max(worst, ((out.float() - whole[last].float()).norm() / whole[last].float().norm()).item())
    print(f"{steps} tokens for {len(lens)} requests after prompts of {lens}: absorbed against expanded, "
          f"relative difference {worst:.2e}")
    continue_forked()
    return worst


if __name__ == "__main__":
    main()
