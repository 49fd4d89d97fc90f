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
FP32 = torch.finfo(torch.float32)
INT_MAX = 2 ** 31 - 1
SHARED_KEYS = 8192   # packed keys below which latent_fwd has no use for a workspace

_FLOAT_FLAGS = {torch.bfloat16: 0, torch.float16: KDA_FLAG_FP16}


# Decode steps are a few microseconds of GPU time: each function tests its
# arguments in one plain condition, and only where that fails goes through the
# checks below, which say what is wrong.
def _check(name: str, t, dtype, shape) -> None:
    """``shape``: the wanted sizes, None where any size goes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        raise ValueError(f"{name} must have shape [{want}], got {tuple(t.shape)}")


def _check_int(name: str, value) -> None:
    """The C entries take 32 bits, and ctypes drops the others."""
    if not -INT_MAX <= value <= INT_MAX or value != int(value):
        raise ValueError(f"{name} must be a whole number of 32 bits, got {value}")


def _float_flag(name: str, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    flag = _FLOAT_FLAGS.get(t.dtype)
    if flag is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return flag


def _together(index: int, *tensors) -> bool:
    """Whether all of them (None aside) are on CUDA device ``index``."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            return False
    return index >= 0


def _same_device(index: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on the same device: got cuda:{index} and {t.device}")


def _check_workspace(workspace, index: int) -> None:
    """The kernels write through its pointer, so it has to be the GPU's own memory in one piece."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}, got one on {workspace.device}")


def _status_workspace(workspace, index: int) -> Optional[int]:
    if workspace is None:
        return None
    _check_workspace(workspace, index)
    if workspace.numel() * workspace.element_size() < STATUS_BYTES:
        raise ValueError(f"workspace must have at least {STATUS_BYTES} bytes")
    return workspace.data_ptr()


def _scratch(workspace, need: int, index: int, device) -> torch.Tensor:
    """The caller's workspace, or a fresh one where there is none or it is too small (see ``_hand_back``)."""
    if workspace is not None:
        _check_workspace(workspace, index)
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return torch.empty(max(need, STATUS_BYTES), dtype=torch.uint8, device=device)


def _hand_back(scratch, workspace) -> None:
    """After the launch: what the call recorded goes to the caller's workspace where a larger one stood in for it."""
    if workspace is not None and workspace is not scratch:
        own = workspace.view(-1).view(torch.uint8)
        count = min(STATUS_BYTES, own.numel())
        own[:count].copy_(scratch[:count])


def _scale(scale) -> float:
    """The C entries take what is not above zero for the default."""
    if scale is None:
        return -1.0
    if not FP32.tiny <= scale <= FP32.max:
        raise ValueError(f"scale must be a positive finite fp32 number or None, got {scale}")
    return float(scale)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _elsewhere(index: int, fn, *args):
    """``fn`` again, with device ``index`` current."""
    with torch.cuda.device(index):
        return fn(*args)


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raise(rc: int, name: str) -> None:
    if rc != 0:
        raise KdaError(rc, name)


def _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k):
    """Checks what forward and backward share: (q, kv, k_pe, its row stride, N, flags)."""
    flags = _float_flag("q", q)
    dtype, packed = q.dtype, cu_seqlens_q is not None
    if packed != (cu_seqlens_k is not None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k go together")
    try:
        fine = (q.dim() == kv.dim() == 4 and k_pe.dim() == 3 and kv.dtype is k_pe.dtype is dtype
                and q.shape[3] == QUERY_CHANNELS and kv.shape[3] == KEY_CHANNELS + VALUE_CHANNELS
                and k_pe.shape[2] == PE_CHANNELS and q.shape[2] == kv.shape[2] and q.shape[0] == kv.shape[0]
                and k_pe.shape[:2] == kv.shape[:2]
                and (not packed or cu_seqlens_q.dtype is cu_seqlens_k.dtype is torch.int32 and cu_seqlens_q.dim() == 1
                     and cu_seqlens_q.shape == cu_seqlens_k.shape)
                and _together(q.get_device(), kv, k_pe, cu_seqlens_q, cu_seqlens_k))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check("q", q, dtype, (None, None, None, QUERY_CHANNELS))
        _check("kv", kv, dtype, (q.shape[0], None, q.shape[2], KEY_CHANNELS + VALUE_CHANNELS))
        _check("k_pe", k_pe, dtype, (q.shape[0], kv.shape[1], PE_CHANNELS))
        if packed:
            _check("cu_seqlens_q", cu_seqlens_q, torch.int32, (None,))
            _check("cu_seqlens_k", cu_seqlens_k, torch.int32, cu_seqlens_q.shape)
        _same_device(q.get_device(), kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    B, Tk = kv.shape[:2]
    N = B
    if packed:
        N = cu_seqlens_q.shape[0] - 1
        if B != 1 or N < 1:
            raise ValueError("packed sequences need a leading size of 1 and at least one sequence")
        cu_seqlens_q, cu_seqlens_k = cu_seqlens_q.contiguous(), cu_seqlens_k.contiguous()
    q, kv = _aligned(q.contiguous()), _aligned(kv.contiguous())
    # rows of a wider tensor are read in place where the kernels can
    steps = k_pe.stride()
    stride = steps[1] if Tk > 1 else steps[0]
    if (steps[2] != 1 or stride < PE_CHANNELS or stride % 8 or k_pe.data_ptr() % 16
            or (B > 1 and steps[0] != Tk * stride)):
        k_pe = _aligned(k_pe.contiguous())
        stride = PE_CHANNELS
    return q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k


def _aligned(t):
    """The kernels read 16 bytes at a time: a contiguous view that starts elsewhere is copied."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def latent_fwd_workspace_bytes(B: int, Tq: int, Tk: int, H: int, N: int) -> int:
    return int(load_library().kda_latent_fwd_workspace_bytes(B, Tq, Tk, H, N))


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
    ``workspace`` (256-byte aligned) records device-detected faults for
    ``binding.get_status``; with ``latent_fwd_workspace_bytes`` bytes, 256 at
    least, it also serves packed sequences some of which have many more keys
    than the others, for which one is allocated otherwise."""
    q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k = _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    index = q.get_device()
    if index != _current_device():
        return _elsewhere(index, latent_fwd, q, kv, k_pe, scale, causal, cu_seqlens_q, cu_seqlens_k, workspace)
    B, Tq, H, _ = q.shape
    Tk = kv.shape[1]
    o = torch.empty((B, Tq, H, VALUE_CHANNELS), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Tq, H), dtype=torch.float32, device=q.device)
    if workspace is None and cu_seqlens_q is not None and Tk >= SHARED_KEYS:
        need = latent_fwd_workspace_bytes(B, Tq, Tk, H, N)
        if need > STATUS_BYTES:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _raise(load_library().kda_latent_fwd_ws(
        q.data_ptr(), kv.data_ptr(), k_pe.data_ptr(), stride, _scale(scale), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_k), o.data_ptr(), lse.data_ptr(), B, Tq, Tk, H, N, flags | KDA_FLAG_CAUSAL if causal else flags,
        _status_workspace(workspace, index), size, _stream(index)), "kda_latent_fwd")
    return o, lse


def latent_bwd_workspace_bytes(B: int, Tq: int, Tk: int, H: int, N: int) -> int:
    return int(load_library().kda_latent_bwd_workspace_bytes(B, Tq, Tk, H, N))


def latent_bwd(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
               do: torch.Tensor, scale: Optional[float] = None, causal: bool = True,
               cu_seqlens_q: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward of ``latent_fwd`` with the same arguments, its results o and
    lse, and o's gradient ``do``: returns (dq, dkv, dk_pe) in q's type, dk_pe
    summed over the heads.  Deterministic.  ``workspace`` (256-byte aligned)
    has ``latent_bwd_workspace_bytes`` bytes; beside a smaller one another is
    allocated, and the status still goes to it."""
    q, kv, k_pe, stride, N, flags, cu_seqlens_q, cu_seqlens_k = _expanded(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k)
    index = q.get_device()
    B, Tq, H, _ = q.shape
    Tk, dev = kv.shape[1], q.device
    try:
        fine = (o.dtype is do.dtype is q.dtype and lse.dtype is torch.float32 and lse.shape == (B, Tq, H)
                and o.shape == do.shape == (B, Tq, H, VALUE_CHANNELS) and _together(index, o, lse, do))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check("o", o, q.dtype, (B, Tq, H, VALUE_CHANNELS))
        _check("do", do, q.dtype, (B, Tq, H, VALUE_CHANNELS))
        _check("lse", lse, torch.float32, (B, Tq, H))
        _same_device(index, o, lse, do)
    if index != _current_device():
        return _elsewhere(index, latent_bwd, q, kv, k_pe, o, lse, do, scale, causal, cu_seqlens_q, cu_seqlens_k, workspace)
    o, do, lse = _aligned(o.contiguous()), _aligned(do.contiguous()), lse.contiguous()
    need = latent_bwd_workspace_bytes(B, Tq, Tk, H, N)
    scratch = _scratch(workspace, need, index, dev)
    dq = torch.empty_like(q)
    dkv = torch.empty_like(kv)
    dk_pe = torch.empty((B, Tk, PE_CHANNELS), dtype=q.dtype, device=dev)
    _raise(load_library().kda_latent_bwd(
        q.data_ptr(), kv.data_ptr(), k_pe.data_ptr(), stride, o.data_ptr(), lse.data_ptr(), do.data_ptr(),
        _scale(scale), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), dq.data_ptr(), dkv.data_ptr(),
        dk_pe.data_ptr(), B, Tq, Tk, H, N, flags | KDA_FLAG_CAUSAL if causal else flags, scratch.data_ptr(),
        scratch.numel() * scratch.element_size(), _stream(index)), "kda_latent_bwd")
    _hand_back(scratch, workspace)
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
    and -inf.  ``workspace`` as for ``latent_bwd``, with
    ``latent_decode_workspace_bytes`` bytes."""
    flags = _float_flag("q", q)
    dtype = q.dtype
    try:
        fine = (q.dim() == 4 and cache.dim() == 3 and block_table.dim() == 2 and cache.dtype is dtype
                and block_table.dtype is torch.int32 and seq_lens.dtype is torch.int32
                and q.shape[3] == cache.shape[2] == ROW_CHANNELS and seq_lens.shape == block_table.shape[:1] == q.shape[:1]
                and block_table.size(1) <= INT_MAX
                and _together(q.get_device(), cache, block_table, seq_lens))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check("q", q, dtype, (None, None, None, ROW_CHANNELS))
        _check("cache", cache, dtype, (None, None, ROW_CHANNELS))
        _check("block_table", block_table, torch.int32, (q.shape[0], None))
        _check("seq_lens", seq_lens, torch.int32, (q.shape[0],))
        _check_int("block_table's width", block_table.shape[1])
        _same_device(q.get_device(), cache, block_table, seq_lens)
    index = q.get_device()
    if index != _current_device():
        return _elsewhere(index, latent_decode, q, cache, block_table, seq_lens, scale, workspace)
    N, S, H, _ = q.shape
    dev = q.device
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    q, block_table, seq_lens = _aligned(q.contiguous()), block_table.contiguous(), seq_lens.contiguous()
    need = latent_decode_workspace_bytes(N, S, H)
    scratch = _scratch(workspace, need, index, dev)
    o = torch.empty((N, S, H, LATENT_CHANNELS), dtype=q.dtype, device=dev)
    lse = torch.empty((N, S, H), dtype=torch.float32, device=dev)
    _raise(load_library().kda_latent_decode(
        q.data_ptr(), cache.data_ptr(), cache.shape[0], cache.shape[1], block_table.data_ptr(), block_table.shape[1],
        seq_lens.data_ptr(), _scale(scale), o.data_ptr(), lse.data_ptr(), N, S, H, flags,
        scratch.data_ptr(), scratch.numel() * scratch.element_size(), _stream(index)), "kda_latent_decode")
    _hand_back(scratch, workspace)
    return o, lse


def latent_append(rows: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                  norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Write rows [T, 576] (bf16 or fp16) into cache [pages, page_size, 576],
    row t at slot ``slots[t]`` (int64, distinct; a negative one is skipped).
    With ``norm_weight`` [512] the latent channels are RMS-normalised on the
    way.  Returns ``cache``, updated in place."""
    flags = _float_flag("rows", rows)
    dtype = rows.dtype
    try:
        fine = (rows.dim() == 2 and cache.dim() == 3 and cache.dtype is dtype and slots.dtype is torch.int64
                and rows.shape[1] == cache.shape[2] == ROW_CHANNELS and slots.shape == rows.shape[:1]
                and (norm_weight is None or norm_weight.dtype is dtype and norm_weight.shape == (LATENT_CHANNELS,))
                and _together(rows.get_device(), slots, cache, norm_weight))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check("rows", rows, dtype, (None, ROW_CHANNELS))
        _check("slots", slots, torch.int64, (rows.shape[0],))
        _check("cache", cache, dtype, (None, None, ROW_CHANNELS))
        if norm_weight is not None:
            _check("norm_weight", norm_weight, dtype, (LATENT_CHANNELS,))
        _same_device(rows.get_device(), slots, cache, norm_weight)
    index = rows.get_device()
    if index != _current_device():
        return _elsewhere(index, latent_append, rows, slots, cache, norm_weight, eps, workspace)
    T = rows.shape[0]
    if norm_weight is not None:
        norm_weight = _aligned(norm_weight.contiguous())
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    stride = rows.stride(0) if T > 1 else ROW_CHANNELS   # a single row's is whatever it was cut from
    if rows.stride(1) != 1 or stride < ROW_CHANNELS or stride % 8 or rows.data_ptr() % 16:
        rows = _aligned(rows.contiguous())
        stride = ROW_CHANNELS
    slots = slots.contiguous()
    _raise(load_library().kda_latent_append(
        rows.data_ptr(), stride, slots.data_ptr(), _ptr(norm_weight), eps, cache.data_ptr(),
        cache.shape[0] * cache.shape[1], T, flags, _status_workspace(workspace, index), _stream(index)), "kda_latent_append")
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
    try:
        fine = (seq_lens.dtype is new_lens.dtype is block_table.dtype is free_pages.dtype is free_head.dtype is torch.int32
                and seq_lens.dim() == free_pages.dim() == 1 and block_table.dim() == 2 and free_head.shape == (1,)
                and new_lens.shape == seq_lens.shape == block_table.shape[:1]
                and _together(seq_lens.get_device(), new_lens, block_table, free_pages, free_head))
        if fine:
            (N, width), (pages,) = block_table.shape, free_pages.shape
            fine = (0 < page_size <= INT_MAX and page_size % 1 == num_tokens % 1 == 0
                    and num_tokens <= INT_MAX and N <= INT_MAX and width <= INT_MAX and pages <= INT_MAX)
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _check_int("page_size", page_size)
        _check_int("num_tokens", num_tokens)
        for name, t in (("seq_lens", seq_lens), ("block_table", block_table), ("free_pages", free_pages)):
            for size in getattr(t, "shape", ()):
                _check_int(f"a size of {name}", size)
        _check("seq_lens", seq_lens, torch.int32, (None,))
        _check("new_lens", new_lens, torch.int32, seq_lens.shape)
        _check("block_table", block_table, torch.int32, (seq_lens.shape[0], None))
        _check("free_pages", free_pages, torch.int32, (None,))
        _check("free_head", free_head, torch.int32, (1,))
        _same_device(seq_lens.get_device(), new_lens, block_table, free_pages, free_head)
        (N, width), (pages,) = block_table.shape, free_pages.shape
    index = seq_lens.get_device()
    if index != _current_device():
        return _elsewhere(index, block_tables, seq_lens, new_lens, block_table, free_pages, free_head, page_size, num_tokens,
                          workspace)
    dev = seq_lens.device
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    # copies are held until the launch: a freed one's memory would go to the next
    seq_lens, new_lens, free_pages = seq_lens.contiguous(), new_lens.contiguous(), free_pages.contiguous()
    slots = torch.empty((num_tokens,), dtype=torch.int64, device=dev)
    cu = torch.empty((N + 1,), dtype=torch.int32, device=dev)
    lens_out, head_out = torch.empty_like(seq_lens), torch.empty_like(free_head)
    _raise(load_library().kda_block_tables(
        seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), width, free_pages.data_ptr(), pages,
        free_head.data_ptr(), int(page_size), slots.data_ptr(), int(num_tokens), cu.data_ptr(), lens_out.data_ptr(),
        head_out.data_ptr(), N, _status_workspace(workspace, index), _stream(index)), "kda_block_tables")
    return slots, cu, lens_out, head_out
