"""A latent-attention layer served and trained: the latent operators together.

``LatentLayer`` holds random weights of one layer of H heads over a hidden
size D (the projections are plain matrix products) and runs

* ``prefill``: block tables for the prompts, their rows into the paged cache,
  attention in the expanded form,
* ``decode``: one token a request: tables, cache row, attention in the
  absorbed form, whose query takes the key projection and whose output the
  value projection,
* ``train``: forward and backward in the expanded form, with the gradient of
  the layer's input.

``python -m chunked_gated_delta_kda_gb300.latent_serving`` prefills a ragged
batch, decodes a few tokens and compares every decoded token's output with the
expanded form over its whole sequence.
"""

from __future__ import annotations

import torch

from . import binding, latent
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
            raise ValueError("prefill sees the new tokens alone: a request with cached ones goes on with decode")
        slots, cu = self._advance(x @ self.w_row.T, new_lens)
        rows = self.cache.view(-1, ROW_CHANNELS)[slots]                 # as the cache holds them
        o, _ = latent.latent_fwd(self._query(x)[None], self._expand(rows)[None], rows[None, :, LATENT_CHANNELS:],
                                 cu_seqlens_q=cu, cu_seqlens_k=cu)
        return o[0]

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
    return worst


if __name__ == "__main__":
    main()
