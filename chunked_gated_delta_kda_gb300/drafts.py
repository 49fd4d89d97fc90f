"""Verification of drafted tokens (argument marshalling only).

``verify_drafts`` says which drafted tokens of a speculative step are accepted
and draws the token behind them; the accepted number is what
``binding.fused_recurrent`` takes as ``num_accepted_tokens``, and what a
request keeps of the step's cached rows (``pages.page_free``).  It runs in a
kernel of ``libkda.so`` (``include/kda.h`` has the contract);
``csrc/kda_marshal.cpp`` calls it, and what that refuses is explained here.  If
the library is missing, the call raises: there is no fallback path.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from .binding import KdaError, load_marshal
from .latent import _check, _check_int, _same_device, _status_workspace

_TYPES = (torch.float32, torch.bfloat16, torch.float16)


def verify_drafts(draft_tokens: torch.Tensor, target_probs: torch.Tensor, uniform: torch.Tensor,
                  draft_probs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Accept drafted tokens so that what comes out is distributed as the target's tokens.

    draft_tokens: int64 [N, S], a negative one ends a sequence's drafts;
    target_probs: fp32, bf16 or fp16 [N, S + 1, V], the target's probabilities
    at each draft's position and behind the last; draft_probs: [N, S, V] of the
    same type, what the drafts were drawn from, or None where the proposer gave
    no probabilities (1 at the draft); both may be slices of wider rows
    (a vocabulary that is padded).  uniform: fp32 [N, S + 1] in [0, 1): draft s
    with token d is accepted where uniform[s] * q(d) < p(d) and all before it
    are; the last number draws the token behind them, from max(p - q, 0) of the
    first draft that is not accepted, or from p behind the last.  Returns
    (tokens int64 [N, S + 1]: the accepted drafts, the token behind them, then
    -1; num_accepted int32 [N], how many those are, 1 to S + 1).
    ``workspace`` (256 bytes, 256-byte aligned) records device-detected faults
    for ``binding.get_status``."""
    out = load_marshal().verify_drafts(draft_tokens, target_probs, uniform, draft_probs, workspace)
    if type(out) is tuple:
        return out
    if out is not None:
        raise KdaError(out, "kda_verify_drafts")
    _check("draft_tokens", draft_tokens, torch.int64, (None, None))
    N, S = draft_tokens.shape
    if not isinstance(target_probs, torch.Tensor):
        raise TypeError("target_probs must be a torch.Tensor")
    if target_probs.dtype not in _TYPES:
        raise TypeError(f"target_probs must be torch.float32, torch.bfloat16 or torch.float16, got {target_probs.dtype}")
    _check("target_probs", target_probs, target_probs.dtype, (N, S + 1, None))
    _check("uniform", uniform, torch.float32, (N, S + 1))
    if draft_probs is not None:
        _check("draft_probs", draft_probs, target_probs.dtype, (N, S, target_probs.shape[2]))
    for size in target_probs.shape:
        _check_int("a size of target_probs", size)
    _same_device(target_probs.get_device(), draft_tokens, uniform, draft_probs)
    _status_workspace(workspace, target_probs.get_device())
    raise ValueError("verify_drafts: an argument must be of another kind")
