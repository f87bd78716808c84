"""The blocks of a paged cache beyond a step's growth (include/specdec_step.h):
requests that go on from others' tokens, blocks moved to the lowest ids, and the
copies that both ask for."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

from . import _check, _on, load_library
from .step import I32, _at, _cache, _device, _on_stream, _word


class Fork(NamedTuple):
    """What kv_fork decides: see include/specdec_step.h."""
    block_table: torch.Tensor  # [B, max_blocks]
    kv_len: torch.Tensor       # [B] tokens
    held: torch.Tensor         # [B] blocks of each request
    shares: torch.Tensor       # [num_blocks] a block's holders beside the first
    ring_state: torch.Tensor   # [2] head and count of the free ring
    copies: torch.Tensor       # [B, 2] blocks to copy, from and to
    count: torch.Tensor        # [1] how many of them


class Compaction(NamedTuple):
    """What kv_compact decides: see include/specdec_step.h."""
    block_table: torch.Tensor  # [B, max_blocks]
    shares: torch.Tensor       # [num_blocks]
    free_ring: torch.Tensor    # [num_blocks]
    ring_state: torch.Tensor   # [2]
    renamed: torch.Tensor      # [num_blocks] a block's new id, -1 for a free one
    copies: torch.Tensor       # [num_blocks // 2, 2] blocks to copy, from and to
    count: torch.Tensor        # [1] how many of them


def page_workspace_bytes(num_blocks: int) -> int:
    return int(load_library().specdec_page_workspace_bytes(num_blocks))


def new_page_workspace(num_blocks: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for kv_fork and kv_compact, of pools
    of up to num_blocks blocks."""
    with _on(stream):
        return torch.zeros(page_workspace_bytes(num_blocks), dtype=torch.uint8, device=device or "cuda")


def _workspace(ws, blocks: int, device, stream, dev: int):
    if ws is None:
        ws = new_page_workspace(blocks, device=device, stream=stream)
    words = ws.numel()
    return ws, _at(ws, words, "workspace", ws.dtype, dev), words * ws.element_size()


def _results(out, kind, sizes, shaped, device, dev: int, stream):
    """The outputs and their addresses: `out`, or parts of one new tensor, of
    which some have a shape."""
    if out is not None:
        return out, [_at(t, n, f"out.{what}", I32, dev) for t, n, what in zip(out, sizes, kind._fields)]
    if stream is None:
        buf = torch.empty(sum(sizes), dtype=I32, device=device)
    else:
        with _on(stream):
            buf = torch.empty(sum(sizes), dtype=I32, device=device)
    at, addresses = buf.data_ptr(), []
    for n in sizes:
        addresses.append(at)
        at += 4 * n
    parts = list(buf.unsafe_split_with_sizes(sizes))
    for i, shape in shaped:
        parts[i] = parts[i].view(shape)
    return kind(*parts), addresses


def kv_fork(block_table: torch.Tensor, kv_len: torch.Tensor, held: torch.Tensor, parent: torch.Tensor,
            shares: torch.Tensor, free_ring: torch.Tensor, ring_state: torch.Tensor, block_size: int,
            accepted_len: Optional[torch.Tensor] = None, keep: Optional[torch.Tensor] = None,
            out: Optional[Fork] = None, workspace: Optional[torch.Tensor] = None,
            error_word: Optional[torch.Tensor] = None, stream=None) -> Fork:
    """Requests [B] that go on from the tokens of old ones [P], their `parent`s
    (see include/specdec_step.h): blocks are shared, part-filled ones that others
    hold are to be copied (kv_copy with the result's copies and count), and those
    without a holder go back to free_ring, in place.  `out` reuses another fork's
    tensors (its shares and ring_state may be the inputs themselves; no other
    output lies on an input).  Without a workspace the call makes one: a loop
    keeps one of its own (new_page_workspace).  Returns a Fork."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [P, max_blocks]")
    P, width = block_table.shape
    B, N = parent.numel(), free_ring.numel()
    dev = _device(block_table, stream)
    fixed = (_at(block_table, P * width, "block_table", I32, dev), _at(kv_len, P, "kv_len", I32, dev),
             _at(accepted_len, P, "accepted_len", I32, dev), _at(held, P, "held", I32, dev), _at(parent, B, "parent", I32, dev),
             _at(keep, B, "keep", I32, dev), _at(shares, N, "shares", I32, dev), _at(free_ring, N, "free_ring", I32, dev),
             _at(ring_state, 2, "ring_state", I32, dev))
    workspace, ws, ws_bytes = _workspace(workspace, N, block_table.device, stream, dev)
    out, to = _results(out, Fork, (B * width, B, B, N, 2, 2 * B, 1), ((0, (B, width)), (5, (B, 2))),
                       block_table.device, dev, stream)
    _check(load_library().kv_fork(P, B, block_size, width, N, *fixed, *to, ws, ws_bytes, _word(error_word, dev),
                                  _on_stream(stream, dev)), "kv_fork")
    return out


def kv_compact(block_table: torch.Tensor, held: torch.Tensor, shares: torch.Tensor, free_ring: torch.Tensor,
               ring_state: torch.Tensor, out: Optional[Compaction] = None, workspace: Optional[torch.Tensor] = None,
               error_word: Optional[torch.Tensor] = None, stream=None) -> Compaction:
    """Names of the blocks in use after they have moved to the lowest ids (see
    include/specdec_step.h); kv_copy with the result's copies and count moves
    them.  Nothing is changed in place, unless `out`, another compaction's
    tensors, names the inputs.  Returns a Compaction."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, width = block_table.shape
    N = free_ring.numel()
    dev = _device(block_table, stream)
    fixed = (_at(block_table, B * width, "block_table", I32, dev), _at(held, B, "held", I32, dev), _at(shares, N, "shares", I32, dev),
             _at(free_ring, N, "free_ring", I32, dev), _at(ring_state, 2, "ring_state", I32, dev))
    workspace, ws, ws_bytes = _workspace(workspace, N, block_table.device, stream, dev)
    moves = N // 2
    out, to = _results(out, Compaction, (B * width, N, N, 2, N, 2 * moves, 1), ((0, (B, width)), (5, (moves, 2))),
                       block_table.device, dev, stream)
    _check(load_library().kv_compact(B, width, N, *fixed, *to, ws, ws_bytes, _word(error_word, dev), _on_stream(stream, dev)),
           "kv_compact")
    return out


class KvLayers:
    """The caches of a model's layers, which share the block tables, as kv_copy
    takes them (kv_layers makes one, once for a model)."""

    def __init__(self, layers: Sequence, stream=None):
        self.tensors = [tuple(x) for x in layers]
        self.device, self.shape, addresses = None, None, []
        for k, v, ks, vs in self.tensors:
            dev = _device(k, stream)
            blocks, H, bs, D, at = _cache(k, v, ks, vs, dev)
            if self.shape is None:
                self.shape, self.device = (blocks, bs, H, D), dev
            elif self.shape != (blocks, bs, H, D):
                raise ValueError("the layers' caches must have one shape")
            if dev < 0:
                raise ValueError("spec-decode tensors must live on a CUDA device")
            addresses += at
        if self.shape is None:
            raise ValueError("kv_layers needs a layer")
        self.pointers = (ctypes.c_void_p * len(addresses))(*addresses)


def kv_layers(layers: Sequence, stream=None) -> KvLayers:
    """A handle of the layers' caches, each (k_cache, v_cache, k_scale,
    v_scale)."""
    return KvLayers(layers, stream)


def kv_copy(copies: torch.Tensor, count: torch.Tensor, layers, stream=None) -> None:
    """Copies blocks, from and to [n, 2] of which `count` [1] hold, in every
    layer's cache (see include/specdec_step.h).  `layers` is kv_layers' handle,
    or the layers' (k_cache, v_cache, k_scale, v_scale) themselves."""
    if not isinstance(layers, KvLayers):
        layers = KvLayers(layers, stream)
    if copies.dim() != 2 or copies.shape[1] != 2:
        raise ValueError("copies must be [n, 2]")
    dev = _device(copies, stream)
    n = copies.shape[0]
    if dev != layers.device:
        raise ValueError("copies and the layers' caches must share a device")
    blocks, bs, H, D = layers.shape
    _check(load_library().kv_copy(_at(copies, 2 * n, "copies", I32, dev), _at(count, 1, "count", I32, dev), n,
                                  len(layers.tensors), layers.pointers, blocks, bs, H, D, _on_stream(stream, dev)), "kv_copy")
