"""Latent attention and its paged cache (argument marshalling only).

Softmax attention whose keys and values come from one shared row a token (512
latent channels and 64 positional ones), for the full-attention layers of a
decoder that are interleaved with KDA layers:

``latent_fwd`` / ``latent_bwd``  expanded form (prefill and training),
``latent_decode``                absorbed form over the paged cache,
``latent_append``                new tokens' rows into their cache slots,
``block_tables``                 block tables and slot map of a step.

Every step runs in the kernels of ``libkda.so`` (``include/kda.h`` has the
contract); this module checks torch tensors, allocates outputs and workspaces
on the tensors' device and passes pointers and torch's current stream.  If the
library is missing, every call raises: there is no fallback path.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from .binding import KDA_FLAG_CAUSAL, KDA_FLAG_FP16, KdaError, load_library

LATENT_CHANNELS = 512
PE_CHANNELS = 64
ROW_CHANNELS = LATENT_CHANNELS + PE_CHANNELS
KEY_CHANNELS = 128
VALUE_CHANNELS = 128
QUERY_CHANNELS = KEY_CHANNELS + PE_CHANNELS
STATUS_BYTES = 256

_FLOAT_FLAGS = {torch.bfloat16: 0, torch.float16: KDA_FLAG_FP16}


# Decode steps are a few microseconds of GPU time, so the checks below run on
# every call as plain comparisons and only a failed one builds its message.
def _check(name: str, t, dtype, shape) -> None:
    """``shape``: the wanted sizes, None where any size goes."""
    if type(t) is torch.Tensor or isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.is_cuda:
            got = t.shape
            if len(got) == len(shape):
                for w, g in zip(shape, got):
                    if w is not None and w != g:
                        break
                else:
                    return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    want = ", ".join("*" if w is None else str(w) for w in shape)
    raise ValueError(f"{name} must have shape [{want}], got {tuple(t.shape)}")


def _float_flag(name: str, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    flag = _FLOAT_FLAGS.get(t.dtype)
    if flag is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return flag


def _same_device(index: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on the same device: got cuda:{index} and {t.device}")


def _status_workspace(workspace) -> Optional[int]:
    if workspace is None:
        return None
    if workspace.numel() * workspace.element_size() < STATUS_BYTES:
        raise ValueError(f"workspace must have at least {STATUS_BYTES} bytes")
    return workspace.data_ptr()


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(name: str, index: int, *args) -> None:
    """The C entry point on torch's current stream of device ``index``."""
    fn = getattr(load_library(), name)
    if index == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise KdaError(rc, name)


def _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k):
    """Checks what forward and backward share: (q, kv, k_pe, its row stride, N, flags)."""
    flags = _float_flag("q", q)
    _check("q", q, q.dtype, (None, None, None, QUERY_CHANNELS))
    B, _, H, _ = q.shape
    _check("kv", kv, q.dtype, (B, None, H, KEY_CHANNELS + VALUE_CHANNELS))
    Tk = kv.shape[1]
    _check("k_pe", k_pe, q.dtype, (B, Tk, PE_CHANNELS))
    if (cu_seqlens_q is None) != (cu_seqlens_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k go together")
    N = B
    if cu_seqlens_q is not None:
        _check("cu_seqlens_q", cu_seqlens_q, torch.int32, (None,))
        N = cu_seqlens_q.shape[0] - 1
        _check("cu_seqlens_k", cu_seqlens_k, torch.int32, (N + 1,))
        if B != 1 or N < 1:
            raise ValueError("packed sequences need a leading size of 1 and at least one sequence")
        cu_seqlens_q, cu_seqlens_k = cu_seqlens_q.contiguous(), cu_seqlens_k.contiguous()
    _same_device(q.get_device(), kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    q, kv = _aligned(q.contiguous()), _aligned(kv.contiguous())
    # rows of a wider tensor are read in place where the kernels can
    stride = k_pe.stride(1) if Tk > 1 else k_pe.stride(0)
    if (k_pe.stride(2) != 1 or stride < PE_CHANNELS or stride % 8 or k_pe.data_ptr() % 16
            or (B > 1 and k_pe.stride(0) != Tk * stride)):
        k_pe = _aligned(k_pe.contiguous())
        stride = PE_CHANNELS
    return q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k


def _aligned(t):
    """The kernels read 16 bytes at a time: a contiguous view that starts elsewhere is copied."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def latent_fwd(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, scale: Optional[float] = None,
               causal: bool = True, cu_seqlens_q: Optional[torch.Tensor] = None,
               cu_seqlens_k: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Latent attention in its expanded form.

    q: bf16 or fp16 [B, Tq, H, 128 + 64]; kv: [B, Tk, H, 128 + 128], the
    expanded keys and values; k_pe: [B, Tk, 64], the positional key that all
    heads share (a slice of wider rows is read in place); cu_seqlens_q and
    cu_seqlens_k: int32 [N + 1] on the device (packed sequences, B == 1) or
    both None.  With ``causal`` query i of a sequence sees the keys up to
    i + Lk - Lq.  ``scale`` None means 192**-0.5.  Returns (o [B, Tq, H, 128],
    lse fp32 [B, Tq, H]); a query that sees no key gets 0 and -inf.
    ``workspace`` (256 bytes, 256-byte aligned) records device-detected faults
    for ``binding.get_status``."""
    q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k = _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    B, Tq, H, _ = q.shape
    o = torch.empty((B, Tq, H, VALUE_CHANNELS), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Tq, H), dtype=torch.float32, device=q.device)
    _call("kda_latent_fwd", q.get_device(), _ptr(q), _ptr(kv), _ptr(k_pe), stride, float(-1.0 if scale is None else scale),
          _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(o), _ptr(lse), B, Tq, kv.shape[1], H, N,
          flags | (KDA_FLAG_CAUSAL if causal else 0), _status_workspace(workspace))
    return o, lse


def latent_bwd_workspace_bytes(B: int, Tq: int, Tk: int, H: int, N: int) -> int:
    return int(load_library().kda_latent_bwd_workspace_bytes(B, Tq, Tk, H, N))


def latent_bwd(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
               do: torch.Tensor, scale: Optional[float] = None, causal: bool = True,
               cu_seqlens_q: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward of ``latent_fwd`` with the same arguments, its results o and
    lse, and o's gradient ``do``: returns (dq, dkv, dk_pe) in q's type, dk_pe
    summed over the heads.  Deterministic."""
    q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k = _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    B, Tq, H, _ = q.shape
    Tk, dev = kv.shape[1], q.device
    _check("o", o, q.dtype, (B, Tq, H, VALUE_CHANNELS))
    _check("do", do, q.dtype, (B, Tq, H, VALUE_CHANNELS))
    _check("lse", lse, torch.float32, (B, Tq, H))
    _same_device(q.get_device(), o, lse, do)
    o, do, lse = _aligned(o.contiguous()), _aligned(do.contiguous()), lse.contiguous()
    need = latent_bwd_workspace_bytes(B, Tq, Tk, H, N)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, STATUS_BYTES), dtype=torch.uint8, device=dev)
    dq = torch.empty_like(q)
    dkv = torch.empty_like(kv)
    dk_pe = torch.empty((B, Tk, PE_CHANNELS), dtype=q.dtype, device=dev)
    _call("kda_latent_bwd", q.get_device(), _ptr(q), _ptr(kv), _ptr(k_pe), stride, _ptr(o), _ptr(lse), _ptr(do),
          float(-1.0 if scale is None else scale), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(dq), _ptr(dkv),
          _ptr(dk_pe), B, Tq, Tk, H, N, flags | (KDA_FLAG_CAUSAL if causal else 0), _ptr(workspace),
          workspace.numel() * workspace.element_size())
    return dq, dkv, dk_pe


def latent_decode_workspace_bytes(N: int, S: int, H: int) -> int:
    return int(load_library().kda_latent_decode_workspace_bytes(N, S, H))


def latent_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Latent attention in its absorbed form over the paged cache.

    q: bf16 or fp16 [N, S, H, 512 + 64], S tokens of each of N sequences, the
    heads' key projection already multiplied in; cache: [pages, page_size, 576]
    (page_size 16, 32, or a multiple of 64); block_table: int32 [N, width];
    seq_lens: int32 [N], the S tokens included: token s sees the first
    seq_lens - S + 1 + s rows.  ``scale`` None means 192**-0.5.  Returns
    (o [N, S, H, 512], lse fp32 [N, S, H]); a token that sees no row gets 0
    and -inf."""
    flags = _float_flag("q", q)
    _check("q", q, q.dtype, (None, None, None, ROW_CHANNELS))
    N, S, H, _ = q.shape
    _check("cache", cache, q.dtype, (None, None, ROW_CHANNELS))
    _check("block_table", block_table, torch.int32, (N, None))
    _check("seq_lens", seq_lens, torch.int32, (N,))
    dev = q.device
    _same_device(q.get_device(), cache, block_table, seq_lens)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    q, block_table, seq_lens = _aligned(q.contiguous()), block_table.contiguous(), seq_lens.contiguous()
    need = latent_decode_workspace_bytes(N, S, H)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, STATUS_BYTES), dtype=torch.uint8, device=dev)
    o = torch.empty((N, S, H, LATENT_CHANNELS), dtype=q.dtype, device=dev)
    lse = torch.empty((N, S, H), dtype=torch.float32, device=dev)
    _call("kda_latent_decode", q.get_device(), _ptr(q), _ptr(cache), cache.shape[0], cache.shape[1], _ptr(block_table),
          block_table.shape[1], _ptr(seq_lens), float(-1.0 if scale is None else scale), _ptr(o), _ptr(lse), N, S, H,
          flags, _ptr(workspace), workspace.numel() * workspace.element_size())
    return o, lse


def latent_append(rows: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                  norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Write rows [T, 576] (bf16 or fp16) into cache [pages, page_size, 576],
    row t at slot ``slots[t]`` (int64, distinct; a negative one is skipped).
    With ``norm_weight`` [512] the latent channels are RMS-normalised on the
    way.  Returns ``cache``, updated in place."""
    flags = _float_flag("rows", rows)
    _check("rows", rows, rows.dtype, (None, ROW_CHANNELS))
    T = rows.shape[0]
    _check("slots", slots, torch.int64, (T,))
    _check("cache", cache, rows.dtype, (None, None, ROW_CHANNELS))
    if norm_weight is not None:
        _check("norm_weight", norm_weight, rows.dtype, (LATENT_CHANNELS,))
        norm_weight = _aligned(norm_weight.contiguous())
    _same_device(rows.get_device(), slots, cache, norm_weight)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    if rows.stride(1) != 1 or rows.stride(0) < ROW_CHANNELS or rows.stride(0) % 8 or rows.data_ptr() % 16:
        rows = _aligned(rows.contiguous())
    slots = slots.contiguous()
    _call("kda_latent_append", rows.get_device(), _ptr(rows), max(rows.stride(0), ROW_CHANNELS), _ptr(slots),
          _ptr(norm_weight), float(eps), _ptr(cache), cache.shape[0] * cache.shape[1], T, flags,
          _status_workspace(workspace))
    return cache


def block_tables(seq_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                 free_head: torch.Tensor, page_size: int, num_tokens: int, workspace: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Block tables and slot map of one step, on the device.

    seq_lens, new_lens: int32 [N], the cached rows of each sequence and the
    tokens it gets; block_table: int32 [N, width], the cells of the pages taken
    now are written in place; free_pages: int32 [F] and free_head: int32 [1],
    the free list and the next entry to take; page_size: a power of two;
    num_tokens: the size of the slot map.  Returns (slot_mapping int64
    [num_tokens], cu_seqlens int32 [N + 1], the new lengths int32 [N], the new
    free_head int32 [1]); the inputs stay as they are."""
    _check("seq_lens", seq_lens, torch.int32, (None,))
    N = seq_lens.shape[0]
    _check("new_lens", new_lens, torch.int32, (N,))
    _check("block_table", block_table, torch.int32, (N, None))
    _check("free_pages", free_pages, torch.int32, (None,))
    _check("free_head", free_head, torch.int32, (1,))
    dev = seq_lens.device
    _same_device(seq_lens.get_device(), new_lens, block_table, free_pages, free_head)
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    slots = torch.empty((num_tokens,), dtype=torch.int64, device=dev)
    out = torch.empty((2 * N + 2,), dtype=torch.int32, device=dev)
    cu, lens_out, head_out = out.split((N + 1, N, 1))
    # copies are held until the launch: a freed one's memory would go to the next
    seq_lens, new_lens, free_pages = seq_lens.contiguous(), new_lens.contiguous(), free_pages.contiguous()
    _call("kda_block_tables", seq_lens.get_device(), _ptr(seq_lens), _ptr(new_lens), _ptr(block_table),
          block_table.shape[1], _ptr(free_pages), free_pages.shape[0], _ptr(free_head), int(page_size),
          _ptr(slots), int(num_tokens), _ptr(cu), _ptr(lens_out), _ptr(head_out), N,
          _status_workspace(workspace))
    return slots, cu, lens_out, head_out
