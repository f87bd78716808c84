"""The operators of a decode step around the verify call (include/specdec_step.h):
block tables and slot maps, the 8-bit cache's writer, attention over it, and
logit processing.  As in the rest of the package, the functions keep the C
names and only marshal tensors: every computation runs in the library's
kernels, on the current CUDA stream or the one given."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _dtype_code, _need, _on, _one_device, _ptr, _stream, load_library

DEV_ERR_BLOCKS, DEV_ERR_PENALTY = 32, 64
ATTENTION_WORKSPACE_BYTES = 64 << 20
E4M3 = torch.float8_e4m3fn

# Every symbol the header declares.
STEP_EXPORTS = ("kv_block_step", "kv_append", "spec_attention", "spec_process_logits")


def _error_word(t: Optional[torch.Tensor]):
    if t is not None and t.numel() * t.element_size() < 4:
        raise ValueError("error_word must hold at least 4 bytes")
    return _ptr(t)


class BlockStep(NamedTuple):
    """What kv_block_step decides: see include/specdec_step.h."""
    kv_len: torch.Tensor       # [B] tokens kept, before the new ones
    held: torch.Tensor         # [B] blocks of each request
    ring_state: torch.Tensor   # [2] head and count of the free ring
    cu_tokens: torch.Tensor    # [B + 1] prefix sums of the new tokens
    cu_blocks: torch.Tensor    # [B + 1] prefix sums of the blocks taken
    slot_map: torch.Tensor     # [capacity] slot of each new token, -1 past the last
    positions: torch.Tensor    # [capacity] position of each new token, -1 past the last


def declare(L) -> None:
    """Argument types of this module's C functions."""
    P, i32, i64, sz, f32, ci = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float,
                                ctypes.c_int)
    L.kv_block_step.argtypes = [i32] * 4 + [P] * 14 + [i32, P, P]
    L.kv_append.argtypes = [P, P, ci, i32, i32, i32, i64, i64, i64, i64, P, i32, i32, P, P, P, P, P]
    L.spec_attention.argtypes = [P, i64, i32, i32, i32, i32, i32, P, P, P, i32, i32, i32, P, P, P, P, f32, P, P, sz, P]
    L.spec_process_logits.argtypes = [P, P, ci, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P, P, P, i32, P, i32, P, P, P]
    for name in STEP_EXPORTS:
        getattr(L, name).restype = ci


def kv_block_step(block_table: torch.Tensor, kv_len: torch.Tensor, held: torch.Tensor, new_tokens: torch.Tensor,
                  free_ring: torch.Tensor, ring_state: torch.Tensor, block_size: int, capacity: int,
                  accepted_len: Optional[torch.Tensor] = None, out: Optional[BlockStep] = None,
                  error_word: Optional[torch.Tensor] = None, stream=None) -> BlockStep:
    """Blocks and slots of the next tokens from the lengths that the last step
    left on the device (see include/specdec_step.h).  block_table
    [B, max_blocks] and free_ring [num_blocks] are updated in place; `out`
    reuses another step's tensors (its kv_len, held and ring_state may be the
    inputs themselves).  Returns a BlockStep."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    blocks = free_ring.numel()
    i32 = torch.int32
    _need(block_table, B * width, "block_table", i32)
    _need(kv_len, B, "kv_len", i32)
    _need(held, B, "held", i32)
    _need(new_tokens, B, "new_tokens", i32)
    _need(accepted_len, B, "accepted_len", i32)
    _need(free_ring, blocks, "free_ring", i32)
    _need(ring_state, 2, "ring_state", i32)
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    if out is None:
        with _on(stream):
            # one allocation, each part on a 16-byte boundary
            sizes = (B, B, 2, B + 1, B + 1, capacity, capacity)
            buf = torch.empty(sum((n + 3) // 4 * 4 for n in sizes), dtype=i32, device=block_table.device)
            parts, at = [], 0
            for n in sizes:
                parts.append(buf[at:at + n])
                at += (n + 3) // 4 * 4
            out = BlockStep(*parts)
    else:
        for t, n, what in zip(out, (B, B, 2, B + 1, B + 1, capacity, capacity), BlockStep._fields):
            _need(t, n, f"out.{what}", i32)
    _one_device(block_table, kv_len, held, new_tokens, accepted_len, free_ring, ring_state, *out, error_word,
                stream=stream)
    _check(load_library().kv_block_step(
        B, block_size, width, blocks, _ptr(kv_len), _ptr(accepted_len), _ptr(new_tokens), _ptr(held),
        _ptr(block_table), _ptr(free_ring), _ptr(ring_state), _ptr(out.kv_len), _ptr(out.held), _ptr(out.ring_state),
        _ptr(out.cu_tokens), _ptr(out.cu_blocks), _ptr(out.slot_map), _ptr(out.positions), capacity,
        _error_word(error_word), _stream(stream)), "kv_block_step")
    return out


def _cache(k_cache, v_cache, k_scale, v_scale):
    """Shape (num_blocks, H, block_size, D) of a cache after its checks."""
    if k_cache.dim() != 4 or k_cache.dtype != E4M3 or v_cache.dtype != E4M3:
        raise TypeError("k_cache and v_cache must be [num_blocks, H, block_size, D] of float8_e4m3fn")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    blocks, H, bs, D = k_cache.shape
    _need(k_scale, blocks * H, "k_scale", torch.float32)
    _need(v_scale, blocks * H, "v_scale", torch.float32)
    return blocks, H, bs, D


def _strided(x: torch.Tensor, what: str):
    """Pointer and the strides of tokens and heads of [T, H, D] rows whose D
    values are contiguous."""
    if not x.is_cuda:
        raise ValueError("spec-decode tensors must live on a CUDA device")
    if x.stride(2) != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return ctypes.c_void_p(x.data_ptr()), x.stride(0), x.stride(1)


def kv_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              k_scale: torch.Tensor, v_scale: torch.Tensor, stream=None) -> None:
    """Writes the keys and values [T, H, D] (bf16 or fp32; views of a fused
    projection will do) of new tokens into the cache at slot_map [T] (see
    include/specdec_step.h)."""
    blocks, H, bs, D = _cache(k_cache, v_cache, k_scale, v_scale)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1:] != (H, D):
        raise ValueError("k and v must be [T, H, D] with the cache's H and D")
    if v.dtype != k.dtype:
        raise TypeError("k and v must have one dtype")
    T = k.shape[0]
    _need(slot_map, T, "slot_map", torch.int32)
    _one_device(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=stream)
    kp, kt, kh = _strided(k, "k")
    vp, vt, vh = _strided(v, "v")
    _check(load_library().kv_append(kp, vp, _dtype_code(k), T, H, D, kt, kh, vt, vh, _ptr(slot_map), blocks, bs,
                                    _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _stream(stream)),
           "kv_append")


def new_attention_workspace(device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for spec_attention."""
    with _on(stream):
        return torch.zeros(ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device=device or "cuda")


def spec_attention(q: torch.Tensor, cu_tokens: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the new tokens' queries [T, Hq, D] (bf16) over the cache,
    causal among the new tokens (see include/specdec_step.h).  `scale`
    defaults to 1 / sqrt(D).  Returns [T, Hq, D] bf16."""
    blocks, H, bs, D = _cache(k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != D or q.dtype != torch.bfloat16:
        raise TypeError("q must be [T, Hq, D] of bfloat16 with the cache's D")
    T, Hq, _ = q.shape
    B = kv_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    width = block_table.shape[1]
    _need(cu_tokens, B + 1, "cu_tokens", torch.int32)
    _need(kv_len, B, "kv_len", torch.int32)
    _need(block_table, B * width, "block_table", torch.int32)
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    if out is None:
        with _on(stream):
            out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must be [T, Hq, D]")
    _need(out, T * Hq * D, "out", torch.bfloat16)
    if workspace is None:
        workspace = new_attention_workspace(device=q.device, stream=stream)
    _one_device(q, cu_tokens, kv_len, block_table, k_cache, v_cache, k_scale, v_scale, out, workspace, stream=stream)
    qp, qt, qh = _strided(q, "q")
    if qh != D and Hq > 1:
        raise ValueError("the heads of q must be contiguous")
    _check(load_library().spec_attention(qp, qt if T > 1 else Hq * D, T, Hq, H, D, B, _ptr(cu_tokens), _ptr(kv_len),
                                         _ptr(block_table), width, blocks, bs, _ptr(k_cache), _ptr(v_cache),
                                         _ptr(k_scale), _ptr(v_scale), 0.0 if scale is None else float(scale),
                                         _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "spec_attention")
    return out


def spec_process_logits(logits: torch.Tensor, history: Optional[torch.Tensor] = None,
                        prompt_len: Optional[torch.Tensor] = None, history_len: Optional[torch.Tensor] = None,
                        draft_tokens: Optional[torch.Tensor] = None, draft_len: Optional[torch.Tensor] = None,
                        repetition: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                        frequency: Optional[torch.Tensor] = None, bias_offsets: Optional[torch.Tensor] = None,
                        bias_ids: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                        mask: Optional[torch.Tensor] = None, mask_rows: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits [B, n_max+1, V] (see
    include/specdec_step.h).  `out` defaults to `logits` itself.  Returns
    `out`."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, n_max+1, V]")
    B, rows, V = logits.shape
    n_max = rows - 1
    i32, f32 = torch.int32, torch.float32
    if out is None:
        out = logits
    elif out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must be of logits' shape and dtype")
    S = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history must be [B, S]")
        S = history.shape[1]
        _need(history, B * S, "history", i32)
        if prompt_len is None or history_len is None:
            raise ValueError("history needs prompt_len and history_len")
        _need(prompt_len, B, "prompt_len", i32)
        _need(history_len, B, "history_len", i32)
    if n_max > 0 and draft_tokens is None:
        raise ValueError("rows after the first need draft_tokens")
    _need(draft_tokens, B * n_max, "draft_tokens", i32)
    _need(draft_len, B, "draft_len", i32)
    for t, what in ((repetition, "repetition"), (presence, "presence"), (frequency, "frequency")):
        _need(t, B, what, f32)
    num_bias = 0
    if bias_offsets is not None:
        if bias_ids is None or bias_values is None:
            raise ValueError("bias_offsets needs bias_ids and bias_values")
        _need(bias_offsets, B + 1, "bias_offsets", i32)
        num_bias = bias_ids.numel()
        _need(bias_ids, num_bias, "bias_ids", i32)
        _need(bias_values, num_bias, "bias_values", f32)
    masks = 0
    if (mask is None) != (mask_rows is None):
        raise ValueError("mask and mask_rows go together")
    if mask is not None:
        if mask.dim() != 2 or mask.shape[1] != (V + 31) // 32:
            raise ValueError("mask must be [masks, ceil(V / 32)]")
        masks = mask.shape[0]
        _need(mask, masks * mask.shape[1], "mask", i32)
        _need(mask_rows, B * rows, "mask_rows", i32)
        if masks == 0:
            mask = mask_rows = None
    _one_device(logits, out, history, prompt_len, history_len, draft_tokens, draft_len, repetition, presence, frequency,
                bias_offsets, bias_ids, bias_values, mask, mask_rows, error_word, stream=stream)
    _check(load_library().spec_process_logits(
        _ptr(logits), _ptr(out), _dtype_code(logits), B, n_max, V, _ptr(history) if S else None, S,
        _ptr(prompt_len) if S else None, _ptr(history_len) if S else None, _ptr(draft_tokens), _ptr(draft_len),
        _ptr(repetition), _ptr(presence), _ptr(frequency), _ptr(bias_offsets), _ptr(bias_ids), _ptr(bias_values),
        num_bias, _ptr(mask), masks, _ptr(mask_rows), _error_word(error_word), _stream(stream)), "spec_process_logits")
    return out
