"""The operators of a decode step around the verify call (include/specdec_step.h):
block tables and slot maps, the 8-bit cache's writer, attention over it, logit
processing, sampling and rotary positions (forks and moves of the cache's blocks
are in pages.py).  As in the rest of the package, the functions keep the C
names and only marshal tensors: every computation runs in the library's
kernels, on the current CUDA stream or the one given."""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _check, _dtype_code, _need, _on, _one_device, _ptr, _stream, load_library

# A decode step's calls last some microseconds on the GPU: their checks use one
# look at each tensor, and the long way round only to say what is wrong.
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16

DEV_ERR_BLOCKS, DEV_ERR_PENALTY, DEV_ERR_SAMPLE = 32, 64, 128
ATTENTION_WORKSPACE_BYTES = 64 << 20
E4M3 = torch.float8_e4m3fn

# Every symbol the header declares.
STEP_EXPORTS = ("kv_block_step", "kv_block_step_shared", "kv_append", "spec_attention", "spec_process_logits", "spec_sample", "spec_rotary",
                "kv_fork", "kv_compact", "kv_copy")


def _device(t: torch.Tensor, stream) -> int:
    """The index of the device of a call's first tensor, which is the current
    one; -2 where it is on none (after the other checks _on_stream says so)."""
    dev = t.get_device()
    if dev < 0:
        return -2
    if stream is not None or dev != _current_device():
        _one_device(t, stream=stream)
    return dev


def _at(t: Optional[torch.Tensor], n: int, what: str, dtype, dev: int):
    """Address of a contiguous tensor of n elements of dtype on a device."""
    if t is None:
        return None
    if t.numel() != n or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _need(t, n, what, dtype)
        if dev >= 0:
            _ptr(t)
            _one_device(t)
    return t.data_ptr()


def _word(t: Optional[torch.Tensor], dev: int):
    if t is None:
        return None
    if t.numel() * t.element_size() < 4:
        raise ValueError("error_word must hold at least 4 bytes")
    return _at(t, t.numel(), "error_word", t.dtype, dev)


def _on_stream(stream, dev: int):
    if dev < 0:
        raise ValueError("spec-decode tensors must live on a CUDA device")
    return _current_stream(dev) if stream is None else _stream(stream)


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
    if hasattr(L, "kv_block_step_shared"):
        L.kv_block_step_shared.argtypes = [i32] * 4 + [P] * 15 + [i32, P, P]
    L.kv_append.argtypes = [P, P, ci, i32, i32, i32, i64, i64, i64, i64, P, i32, i32, P, P, P, P, P]
    L.spec_attention.argtypes = [P, i64, i32, i32, i32, i32, i32, P, P, P, i32, i32, i32, P, P, P, P, f32, P, P, sz, P]
    L.spec_process_logits.argtypes = [P, P, ci, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P, P, P, i32, P, i32, P, P, P]
    if hasattr(L, "spec_sample"):
        L.spec_sample.argtypes = [P, P, ci, i32, i32, i32, P, P, P, P, P, P, P, P, P]
        L.spec_rotary.argtypes = [P, P, ci, i32, i32, i32, i32, i64, i64, i64, i64, P, P, i32, i32, f32, P, i64, i64, P, i64, i64, P]
        L.kv_fork.argtypes = [i32] * 5 + [P] * 17 + [sz, P, P]
        L.kv_compact.argtypes = [i32] * 3 + [P] * 13 + [sz, P, P]
        L.kv_copy.argtypes = [P, P, i32, i32, P, i32, i32, i32, i32, P]
        L.specdec_page_workspace_bytes.argtypes = [i32]
        L.specdec_page_workspace_bytes.restype = sz
    for name in STEP_EXPORTS:
        if hasattr(L, name):
            getattr(L, name).restype = ci


def kv_block_step(block_table: torch.Tensor, kv_len: torch.Tensor, held: torch.Tensor, new_tokens: torch.Tensor,
                  free_ring: torch.Tensor, ring_state: torch.Tensor, block_size: int, capacity: int,
                  accepted_len: Optional[torch.Tensor] = None, out: Optional[BlockStep] = None,
                  error_word: Optional[torch.Tensor] = None, stream=None, shares: Optional[torch.Tensor] = None) -> BlockStep:
    """Blocks and slots of the next tokens from the lengths that the last step
    left on the device (see include/specdec_step.h).  block_table
    [B, max_blocks] and free_ring [num_blocks] are updated in place; `out`
    reuses another step's tensors (its kv_len, held and ring_state may be the
    inputs themselves).  With `shares` [num_blocks] (kv_fork's), requests that
    would write or give back a block that others hold are refused.  Returns a
    BlockStep."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    blocks = free_ring.numel()
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    dev = _device(block_table, stream)
    fixed = (_at(kv_len, B, "kv_len", I32, dev), _at(accepted_len, B, "accepted_len", I32, dev),
             _at(new_tokens, B, "new_tokens", I32, dev), _at(held, B, "held", I32, dev),
             _at(block_table, B * width, "block_table", I32, dev), _at(free_ring, blocks, "free_ring", I32, dev),
             _at(ring_state, 2, "ring_state", I32, dev))
    if out is None:
        # one allocation, in the fields' order (slot_map lies on 16 bytes)
        with _on(stream):
            buf = torch.empty(4 * B + 4 + 2 * capacity, dtype=I32, device=block_table.device)
        out = BlockStep._make(buf.unsafe_split_with_sizes((B, B, 2, B + 1, B + 1, capacity, capacity)))
        at = buf.data_ptr()
        slots = at + 16 * B + 16
        results = (at, at + 4 * B, at + 8 * B, at + 8 * B + 8, at + 12 * B + 12, slots, slots + 4 * capacity)
    else:
        results = [_at(t, n, f"out.{what}", I32, dev)
                   for t, n, what in zip(out, (B, B, 2, B + 1, B + 1, capacity, capacity), BlockStep._fields)]
    last = (capacity, _word(error_word, dev), _on_stream(stream, dev))
    if shares is None:
        _check(load_library().kv_block_step(B, block_size, width, blocks, *fixed, *results, *last), "kv_block_step")
    else:
        _check(load_library().kv_block_step_shared(B, block_size, width, blocks, *fixed, _at(shares, blocks, "shares", I32, dev), *results,
                                                   *last), "kv_block_step_shared")
    return out


def _cache(k_cache, v_cache, k_scale, v_scale, dev: int):
    """Shape (num_blocks, H, block_size, D) of a cache and the addresses of
    its four parts, after its checks."""
    if k_cache.dim() != 4 or k_cache.dtype is not E4M3 or v_cache.dtype is not E4M3:
        raise TypeError("k_cache and v_cache must be [num_blocks, H, block_size, D] of float8_e4m3fn")
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape")
    blocks, H, bs, D = shape
    n = blocks * H
    return blocks, H, bs, D, (_at(k_cache, n * bs * D, "k_cache", E4M3, dev), _at(v_cache, n * bs * D, "v_cache", E4M3, dev),
                              _at(k_scale, n, "k_scale", F32, dev), _at(v_scale, n, "v_scale", F32, dev))


def _strided(x: torch.Tensor, what: str, dev: int):
    """Address and the strides of tokens and heads of [T, H, D] rows whose D
    values are contiguous."""
    if x.get_device() != dev and dev >= 0:
        if not x.is_cuda:
            raise ValueError("spec-decode tensors must live on a CUDA device")
        _one_device(x)
    token, head, one = x.stride()
    if one != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    T, H, D = x.shape
    # (one token, or one head, is as far from the next as it would be if contiguous)
    head = head if H > 1 else D
    return x.data_ptr(), token if T > 1 else H * head, head


def kv_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              k_scale: torch.Tensor, v_scale: torch.Tensor, stream=None) -> None:
    """Writes the keys and values [T, H, D] (bf16 or fp32; views of a fused
    projection will do) of new tokens into the cache at slot_map [T] (see
    include/specdec_step.h)."""
    dev = _device(k, stream)
    blocks, H, bs, D, cache = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1:] != (H, D):
        raise ValueError("k and v must be [T, H, D] with the cache's H and D")
    if v.dtype != k.dtype:
        raise TypeError("k and v must have one dtype")
    T = k.shape[0]
    slots = _at(slot_map, T, "slot_map", I32, dev)
    kp, kt, kh = _strided(k, "k", dev)
    vp, vt, vh = _strided(v, "v", dev)
    _check(load_library().kv_append(kp, vp, _dtype_code(k), T, H, D, kt, kh, vt, vh, slots, blocks, bs, *cache,
                                    _on_stream(stream, dev)), "kv_append")


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
    defaults to 1 / sqrt(D).  Without a workspace the call makes one, 64 MB
    filled with zeros every time: a loop keeps one of its own
    (new_attention_workspace).  Returns [T, Hq, D] bf16."""
    dev = _device(q, stream)
    blocks, H, bs, D, cache = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3 or q.shape[2] != D or q.dtype is not BF16:
        raise TypeError("q must be [T, Hq, D] of bfloat16 with the cache's D")
    T, Hq, _ = q.shape
    B = kv_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    width = block_table.shape[1]
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    if out is None:
        with _on(stream):
            out = torch.empty(T, Hq, D, dtype=BF16, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must be [T, Hq, D]")
    lengths = (_at(cu_tokens, B + 1, "cu_tokens", I32, dev), _at(kv_len, B, "kv_len", I32, dev),
               _at(block_table, B * width, "block_table", I32, dev))
    to = _at(out, T * Hq * D, "out", BF16, dev)
    if workspace is None:
        workspace = new_attention_workspace(device=q.device, stream=stream)
    qp, qt, qh = _strided(q, "q", dev)
    if qh != D:
        raise ValueError("the heads of q must be contiguous")
    words = workspace.numel()
    size = words * workspace.element_size()
    _check(load_library().spec_attention(qp, qt, T, Hq, H, D, B, *lengths, width, blocks, bs,
                                         *cache, 0.0 if scale is None else float(scale), to,
                                         _at(workspace, words, "workspace", workspace.dtype, dev), size,
                                         _on_stream(stream, dev)), "spec_attention")
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
    dev = _device(logits, stream)
    dtype = logits.dtype
    at = _at(logits, B * rows * V, "logits", dtype, dev)
    if out is None or out is logits:
        out, to = logits, at
    else:
        if out.shape != logits.shape or out.dtype != dtype:
            raise ValueError("out must be of logits' shape and dtype")
        to = _at(out, B * rows * V, "out", dtype, dev)
    S = 0
    past = (None, 0, None, None)
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history must be [B, S]")
        S = history.shape[1]
        if prompt_len is None or history_len is None:
            raise ValueError("history needs prompt_len and history_len")
        lens = _at(prompt_len, B, "prompt_len", I32, dev), _at(history_len, B, "history_len", I32, dev)
        ids = _at(history, B * S, "history", I32, dev)
        if S:
            past = (ids, S, *lens)
    if n_max > 0 and draft_tokens is None:
        raise ValueError("rows after the first need draft_tokens")
    drafts = (_at(draft_tokens, B * n_max, "draft_tokens", I32, dev), _at(draft_len, B, "draft_len", I32, dev))
    penalties = (_at(repetition, B, "repetition", F32, dev), _at(presence, B, "presence", F32, dev),
                 _at(frequency, B, "frequency", F32, dev))
    num_bias = 0
    biases = (None, None, None)
    if bias_offsets is not None:
        if bias_ids is None or bias_values is None:
            raise ValueError("bias_offsets needs bias_ids and bias_values")
        num_bias = bias_ids.numel()
        biases = (_at(bias_offsets, B + 1, "bias_offsets", I32, dev), _at(bias_ids, num_bias, "bias_ids", I32, dev),
                  _at(bias_values, num_bias, "bias_values", F32, dev))
    if (mask is None) != (mask_rows is None):
        raise ValueError("mask and mask_rows go together")
    masks, words, named = 0, None, None
    if mask is not None:
        if mask.dim() != 2 or mask.shape[1] != (V + 31) // 32:
            raise ValueError("mask must be [masks, ceil(V / 32)]")
        masks = mask.shape[0]
        words, named = _at(mask, masks * mask.shape[1], "mask", I32, dev), _at(mask_rows, B * rows, "mask_rows", I32, dev)
        if masks == 0:
            words = named = None
    _check(load_library().spec_process_logits(at, to, _dtype_code(logits), B, n_max, V, *past, *drafts, *penalties,
                                              *biases, num_bias, words, masks, named, _word(error_word, dev),
                                              _on_stream(stream, dev)), "spec_process_logits")
    return out


def spec_sample(logits: torch.Tensor, temperature: Optional[torch.Tensor] = None, top_k: Optional[torch.Tensor] = None,
                top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
                uniform: Optional[torch.Tensor] = None, draft_len: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
                error_word: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Truncated sampling on logits [B, n_max+1, V] (see include/specdec_step.h).
    With `uniform` [B, n_max+1], random numbers in [0, 1), a token of each row
    is drawn; with `out` (may be `logits`) the rows are cut to what may be
    drawn, as spec_verify reads them.  Returns the tokens [B, n_max+1], int32
    (`tokens` where given), or None without `uniform`."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, n_max+1, V]")
    B, rows, V = logits.shape
    dev = _device(logits, stream)
    dtype = logits.dtype
    at = _at(logits, B * rows * V, "logits", dtype, dev)
    if out is None:
        to = None
    elif out is logits:
        to = at
    else:
        if out.shape != logits.shape or out.dtype != dtype:
            raise ValueError("out must be of logits' shape and dtype")
        to = _at(out, B * rows * V, "out", dtype, dev)
    if uniform is None:
        if tokens is not None:
            raise ValueError("tokens need uniform")
        if out is None:
            raise ValueError("nothing to do: give uniform, out or both")
    elif tokens is None:
        with _on(stream):
            tokens = torch.empty(B, rows, dtype=I32, device=logits.device)
    _check(load_library().spec_sample(at, to, _dtype_code(logits), B, rows - 1, V, _at(draft_len, B, "draft_len", I32, dev),
                                      _at(temperature, B, "temperature", F32, dev), _at(top_k, B, "top_k", I32, dev),
                                      _at(top_p, B, "top_p", F32, dev), _at(min_p, B, "min_p", F32, dev),
                                      _at(uniform, B * rows, "uniform", F32, dev), _at(tokens, B * rows, "tokens", I32, dev),
                                      _word(error_word, dev), _on_stream(stream, dev)), "spec_sample")
    return tokens


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """Angles a position of each pair, base^(-2 i / rotary_dim), and the factor
    of the turned values, as 64-bit floats.  `scaling` is for contexts longer
    than the training's, by `factor`:

    * ``type="linear"``: all frequencies over the factor;
    * ``type="ntk"``: the base times factor^(rotary_dim / (rotary_dim - 2));
    * ``type="yarn"`` (Peng et al., "YaRN", 2023) with `original` tokens of
      context in training: pairs of more than `fast` (32) turns in it stay, those
      of less than `slow` (1) are scaled, between is a ramp over the pairs, and the
      result is scaled by 0.1 ln(factor) + 1 (or `attention`);
    * ``type="bands"``: pairs of more than `high` turns in `original` tokens stay,
      those of less than `low` are scaled, between is a ramp over the turns."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not (base > 1 and math.isfinite(base)):
        raise ValueError("base must be above 1")
    half = rotary_dim // 2
    freq = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    if scaling is None:
        return freq, 1.0
    kind, rest = scaling.get("type"), {k: v for k, v in scaling.items() if k not in ("type", "factor")}
    by = float(scaling.get("factor", 0.0))
    if not (by >= 1 and math.isfinite(by)):
        raise ValueError("scaling needs a factor of at least 1")
    names = {"linear": (), "ntk": (), "yarn": ("original", "fast", "slow", "attention"), "bands": ("original", "low", "high")}
    if kind not in names or set(rest) - set(names[kind]):
        raise ValueError(f"scaling is linear, ntk, yarn or bands with their own values, got {scaling}")
    if kind == "linear":
        return [f / by for f in freq], 1.0
    if kind == "ntk":
        if rotary_dim == 2:
            raise ValueError("ntk scaling needs more than one pair")
        base = base * by ** (rotary_dim / (rotary_dim - 2.0))
        return [base ** (-2.0 * i / rotary_dim) for i in range(half)], 1.0
    length = float(rest.get("original", 0.0))
    if not (length > 0 and math.isfinite(length)):
        raise ValueError(f"{kind} scaling needs the original context's length")
    if kind == "yarn":
        fast, slow = float(rest.get("fast", 32.0)), float(rest.get("slow", 1.0))
        if not (fast >= slow > 0):
            raise ValueError("yarn scaling needs fast >= slow > 0")
        pair = lambda turns: rotary_dim * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rotary_dim - 1)
        ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(half)]
        given = rest.get("attention")
        factor = 0.1 * math.log(by) + 1.0 if given is None else float(given)
        if not (factor > 0 and math.isfinite(factor)):
            raise ValueError("yarn scaling needs a positive attention")
        return [f * (1.0 - r) + f / by * r for f, r in zip(freq, ramp)], factor
    low, high = float(rest.get("low", 1.0)), float(rest.get("high", 4.0))
    if not (high > low > 0):
        raise ValueError("bands scaling needs high > low > 0")
    keep = [min(max((length * f / (2.0 * math.pi) - low) / (high - low), 0.0), 1.0) for f in freq]
    return [f * r + f / by * (1.0 - r) for f, r in zip(freq, keep)], 1.0


def rotary_turns(rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None, device=None):
    """What spec_rotary takes, made once for a model: `turns` [rotary_dim / 2]
    int64, each pair's frequency (see rotary_frequencies) in 2^-64 of a turn a
    position, and the factor."""
    freq, factor = rotary_frequencies(rotary_dim, base, scaling)
    words = [round(f / (2.0 * math.pi) * 2.0 ** 64) & ((1 << 64) - 1) for f in freq]
    turns = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)
    return turns.to(device or "cuda"), factor


def spec_rotary(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, turns: torch.Tensor,
                layout: str = "half", factor: float = 1.0, q_out: Optional[torch.Tensor] = None,
                k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions of queries [T, Hq, D] and keys [T, H, D] (bf16 or fp32;
    views of a fused projection will do; one of them may be None) at positions
    [T] (see include/specdec_step.h).  `turns` and `factor` are rotary_turns';
    twice the turns' number of each head's values are turned, in pairs (i, i +
    half of them) with ``layout="half"`` or (2 i, 2 i + 1) with
    ``layout="pairs"``.  In place, or into q_out and k_out.  Returns both."""
    one = q if q is not None else k
    if one is None:
        raise ValueError("spec_rotary needs q or k")
    if one.dim() != 3:
        raise ValueError("q and k must be [T, heads, D]")
    if layout not in ("half", "pairs"):
        raise ValueError("layout must be 'half' or 'pairs'")
    dev = _device(one, stream)
    T, _, D = one.shape
    dtype = one.dtype
    sides = []
    for x, y, what in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            if y is not None:
                raise ValueError(f"{what}_out without {what}")
            sides.append((0, (None, 0, 0), (None, 0, 0)))
            continue
        if x.dim() != 3 or x.shape[0] != T or x.shape[2] != D:
            raise ValueError("q and k must be [T, heads, D] with one T and D")
        if x.dtype is not dtype:
            raise TypeError("q and k must have one dtype")
        src = _strided(x, what, dev)
        if y is None or y is x:
            sides.append((x.shape[1], src, src))
            continue
        if y.shape != x.shape:
            raise ValueError(f"{what}_out must be of {what}'s shape")
        if y.dtype is not dtype:
            raise TypeError(f"{what}_out must be of {what}'s dtype")
        sides.append((x.shape[1], src, _strided(y, f"{what}_out", dev)))
    pairs = turns.numel()
    if pairs == 0 or 2 * pairs > D:
        raise ValueError("turns must hold a value for each pair of a head")
    (Hq, (qp, qt, qh), (qo, qot, qoh)), (H, (kp, kt, kh), (ko, kot, koh)) = sides
    _check(load_library().spec_rotary(qp, kp, _dtype_code(one), T, Hq, H, D, qt, qh, kt, kh,
                                      _at(positions, T, "positions", I32, dev), _at(turns, pairs, "turns", torch.int64, dev),
                                      2 * pairs, int(layout == "pairs"), float(factor), qo, qot, qoh, ko, kot, koh,
                                      _on_stream(stream, dev)), "spec_rotary")
    return q if q_out is None else q_out, k if k_out is None else k_out
