"""A step of speculative decoding over a KV cache: the binding of
fd_build_tables, fd_cache_write, fd_tree_decode, fd_tree_decode_paged and
fd_cache_compact (include/fd.h).

    tables = fd_build_tables(lens, new_lens, table, free, free_count, page, num_pages, max_tokens)
    fd_cache_write(k_new, v_new, tables.slot_map, k_pages, v_pages)
    out, lse = fd_tree_decode_paged(q, k_pages, v_pages, table, tables.seq_lens, mask)
    lens = fd_cache_compact(k_pages, v_pages, tables.seq_lens, accepted, accept_lens, tree_len, block_table=table)

Like the package's other functions these only check and marshal arguments;
tensors live on one GPU, outputs are allocated unless they are given.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import (FD_ERR_INVALID_ARG, FD_OK, FdError, FdOptions, _bits, _dtype_code, _kv_code, _lib, _options,
               _ptr, _stream_ptr, fd_workspace_init)

__all__ = ["fd_build_tables", "fd_cache_write", "fd_cache_compact", "fd_tree_workspace_size", "make_tree_workspace",
           "fd_tree_decode", "fd_tree_decode_paged", "Tables", "FD_DEVICE_STATUS_BAD_LENGTH",
           "FD_DEVICE_STATUS_NO_PAGES", "FD_DEVICE_STATUS_BAD_SLOT"]

FD_DEVICE_STATUS_BAD_LENGTH, FD_DEVICE_STATUS_NO_PAGES, FD_DEVICE_STATUS_BAD_SLOT = 0x2, 0x4, 0x8


class Tables(NamedTuple):
    """What fd_build_tables gives back."""
    block_table: torch.Tensor   # [B, max_blocks] int32, the caller's, updated
    slot_map: torch.Tensor      # [max_tokens] int64
    cu_new_lens: torch.Tensor   # [B + 1] int32
    seq_lens: torch.Tensor      # [B] int32, with the new tokens
    held_pages: torch.Tensor    # [B] int32
    free_count: torch.Tensor    # [1] int32


def _dev(t, name, dtype, shape, device):
    """t as a contiguous tensor of this type and shape on the call's device (shape entries None: any)."""
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    return t


def _status(t, device):
    if t is None:
        return None
    if t.dtype not in (torch.int32, torch.uint32) or not t.is_cuda or t.device != device or t.numel() != 1:
        raise ValueError("device_status must be one int32 or uint32 on the call's device")
    return ctypes.c_void_p(t.data_ptr())


def _launch(device, f, *args):
    """Call f with the call's device current (kernels launch on the current device)."""
    if torch.cuda.current_device() == device.index:
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def fd_build_tables(seq_lens, new_lens, block_table, free_pages, free_count, page_size, num_pages, max_tokens,
                    held_pages=None, slot_map=None, device_status=None, stream=None, check=True):
    """Give requests pages and slots for their new tokens (see fd_build_tables in include/fd.h).

    seq_lens, new_lens and held_pages int32 [B]; block_table int32 [B,
    max_blocks], updated in place; free_pages int32 [n], a stack whose first
    free_count (int32 [1]) entries are free; max_tokens the length of the slot
    map (entries behind the last token are -1).  Returns a Tables."""
    i32 = torch.int32
    dev = block_table.device
    B = seq_lens.shape[0]
    _dev(block_table, "block_table", i32, (B, None), dev)
    _dev(seq_lens, "seq_lens", i32, (B,), dev)
    _dev(new_lens, "new_lens", i32, (B,), dev)
    _dev(free_pages, "free_pages", i32, (None,), dev)
    _dev(free_count, "free_count", i32, (1,), dev)
    if held_pages is not None:
        _dev(held_pages, "held_pages", i32, (B,), dev)
    if slot_map is None:
        slot_map = torch.empty(int(max_tokens), dtype=torch.int64, device=dev)
    else:
        _dev(slot_map, "slot_map", torch.int64, (int(max_tokens),), dev)
    cu, lens, held, left = torch.empty(3 * B + 2, dtype=i32, device=dev).split((B + 1, B, B, 1))
    st = _launch(dev, _lib.fd_build_tables, _ptr(seq_lens), _ptr(new_lens), _ptr(held_pages), _ptr(free_pages),
                 _ptr(free_count), free_pages.shape[0], B, int(page_size), int(num_pages), block_table.shape[1],
                 int(max_tokens), _ptr(block_table), _ptr(slot_map), _ptr(cu), _ptr(lens), _ptr(held), _ptr(left),
                 _status(device_status, dev), _stream_ptr(stream, dev))
    if check and st != FD_OK:
        raise FdError(st, "fd_build_tables")
    return Tables(block_table, slot_map, cu, lens, held, left)


def _token_rows(t, name, device):
    """(pointer, stride in elements) of new K or V rows [n, Hkv, D], dense inside a row."""
    if t.dtype not in (torch.bfloat16, torch.float16) or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16 or fp16 CUDA tensor [n, Hkv, D]")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    n, h, d = t.shape
    if t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: a token's heads must be dense (only the token stride is free)")
    return t.stride(0)


def fd_cache_write(k_new, v_new, slot_map, k_cache, v_cache, kv_dtype=None, k_scale=1.0, v_scale=1.0,
                   device_status=None, stream=None, check=True):
    """Write new K/V rows into the cache's slots (see fd_cache_write in include/fd.h).

    k_new, v_new bf16 or fp16 [n, Hkv, D], any token stride that is a multiple
    of 8; slot_map int64 [n] (negative: skip); k_cache, v_cache [..., Hkv, D]
    (pages [num_pages, P, Hkv, D], a contiguous cache [B, S, Hkv, D], or flat
    slots) of the same type, or FP8: float8 tensors, or uint8 codes with
    kv_dtype 'e4m3' / 'e5m2', quantised by k_scale / v_scale."""
    dev = k_cache.device
    ks, vs = _token_rows(k_new, "k_new", dev), _token_rows(v_new, "v_new", dev)
    kv = _kv_code(k_cache, v_cache, kv_dtype)
    n, h, d = k_new.shape
    if v_new.shape != k_new.shape or v_new.dtype != k_new.dtype:
        raise ValueError("k_new and v_new must have one shape and type")
    if k_cache.shape != v_cache.shape or v_cache.device != dev or k_cache.dim() < 3 or tuple(k_cache.shape[-2:]) != (h, d):
        raise ValueError(f"k_cache and v_cache must have one shape [..., {h}, {d}] on one device")
    if kv == 0 and (k_cache.dtype != k_new.dtype or v_cache.dtype != k_new.dtype):
        raise TypeError("a 16-bit cache must be of the new rows' type")
    _dev(slot_map, "slot_map", torch.int64, (n,), dev)
    opts = FdOptions(0, 0, 0, None, None, _dtype_code(k_new, None), kv, float(k_scale), float(v_scale), 1)
    st = _launch(dev, _lib.fd_cache_write, _ptr(k_new), _ptr(v_new), ks, vs, _ptr(slot_map), n, h, d, _ptr(k_cache),
                 _ptr(v_cache), k_cache.numel() // (h * d), ctypes.byref(opts), _status(device_status, dev),
                 _stream_ptr(stream, dev))
    if check and st != FD_OK:
        raise FdError(st, "fd_cache_write")


def fd_cache_compact(k_cache, v_cache, seq_lens, accepted, accept_lens, tree_len, block_table=None, tree_lens=None,
                     seq_lens_out=None, device_status=None, stream=None, check=True):
    """Move the accepted path's rows to the front of the drafted tail, in place
    (see fd_cache_compact in include/fd.h).

    k_cache, v_cache [B, S, Hkv, D], or pages [num_pages, P, Hkv, D] with
    block_table int32 [B, max_blocks], of any type a cache has; seq_lens int32
    [B] with the drafted tokens; accepted int32 [B, max_accept], ascending node
    indices; accept_lens int32 [B]; tree_lens int32 [B] or None (tree_len for
    every request).  Returns the new lengths int32 [B]."""
    dev, i32 = k_cache.device, torch.int32
    B = seq_lens.shape[0]
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != 4 or t.device != dev or t.element_size() > 2:
            raise ValueError(f"{name} must be a contiguous 4-d CUDA tensor of 16-bit or FP8 elements")
    if k_cache.shape != v_cache.shape or k_cache.element_size() != v_cache.element_size():
        raise ValueError("k_cache and v_cache must have one shape and type")
    _dev(seq_lens, "seq_lens", i32, (B,), dev)
    _dev(accepted, "accepted", i32, (B, None), dev)
    _dev(accept_lens, "accept_lens", i32, (B,), dev)
    if tree_lens is not None:
        _dev(tree_lens, "tree_lens", i32, (B,), dev)
    pages, page, h, d = k_cache.shape
    blocks = 0
    if block_table is not None:
        blocks = _dev(block_table, "block_table", i32, (B, None), dev).shape[1]
    elif pages != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {pages}")
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens)
    else:
        _dev(seq_lens_out, "seq_lens_out", i32, (B,), dev)
    opts = FdOptions(0, 0, 0, None, None, 0, 1 if k_cache.element_size() == 1 else 0, 0.0, 0.0, 1)
    st = _launch(dev, _lib.fd_cache_compact, _ptr(k_cache), _ptr(v_cache), _ptr(block_table), blocks, page, pages,
                 _ptr(seq_lens), _ptr(tree_lens), int(tree_len), _ptr(accepted), _ptr(accept_lens), accepted.shape[1],
                 B, h, d, _ptr(seq_lens_out), ctypes.byref(opts), _status(device_status, dev), _stream_ptr(stream, dev))
    if check and st != FD_OK:
        raise FdError(st, "fd_cache_compact")
    return seq_lens_out


def fd_tree_workspace_size(batch, tree_len, num_q_heads, num_kv_heads, head_dim=128) -> int:
    return int(_lib.fd_tree_workspace_size(batch, tree_len, num_q_heads, num_kv_heads, head_dim))


def make_tree_workspace(batch, tree_len, num_q_heads, num_kv_heads, head_dim=128, device="cuda") -> torch.Tensor:
    """Allocate (with torch) and initialise a workspace of fd_tree_decode for this shape."""
    n = fd_tree_workspace_size(batch, tree_len, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_tree_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _launch(ws.device, fd_workspace_init, ws)
    return ws


def _tree_args(q, k, v, tree_mask, tree_lens, seq_lens, seq_lens_host, scale, out, lse, workspace, num_ctas, flags,
               wait_timeout_ns, split_events, dtype, kv_dtype, k_scale, v_scale, block_table):
    """Checks shared by both layouts; the arguments of the C calls that they share."""
    i32 = torch.int32
    _bits(q, "q")
    kv = _kv_code(k, v, kv_dtype)
    dev = q.device
    if q.dim() != 4:
        raise ValueError("q must be [B, tree_len, Hq, D]")
    B, T, hq, d = q.shape
    if k.dim() != 4 or k.shape != v.shape or k.device != dev or v.device != dev or k.shape[3] != d:
        raise ValueError(f"k and v must have one 4-d shape with head_dim {d} on {dev}")
    if kv == 0 and (k.element_size() != 2 or v.element_size() != 2):
        raise TypeError("a 16-bit cache must be of q's type")
    if kv == 0 and torch.float16 in (q.dtype, k.dtype, v.dtype) and torch.bfloat16 in (q.dtype, k.dtype, v.dtype):
        raise TypeError("a 16-bit cache must be of q's type")
    hkv = k.shape[2]
    if tree_lens is not None:
        _dev(tree_lens, "tree_lens", i32, (B,), dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", i32, (B,), dev)
    if block_table is not None:
        _dev(block_table, "block_table", i32, (B, None), dev)
    elif k.shape[0] != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {k.shape[0]}")
    stride, words = 0, (T + 63) // 64
    if tree_mask is not None:
        if tree_mask.dtype not in (torch.int64, torch.uint64):
            raise ValueError("tree_mask must be int64 or uint64 words")
        if tree_mask.dim() == 3:
            _dev(tree_mask, "tree_mask", tree_mask.dtype, (B, T, words), dev)
            stride = T * words
        else:
            _dev(tree_mask, "tree_mask", tree_mask.dtype, (T, words), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, T, hq, d), dtype=torch.float32, device=dev)
    else:
        _dev(out, "out", torch.float32, (B, T, hq, d), dev)
    if lse is None:
        lse = torch.empty((B, T, hq), dtype=torch.float32, device=dev)
    elif lse is not False:
        _dev(lse, "lse", torch.float32, (B, T, hq), dev)
    if workspace is None:
        workspace = make_tree_workspace(B, T, hq, hkv, d, dev)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    lh = None if seq_lens_host is None else seq_lens_host.to(torch.int32).contiguous().cpu()
    if lh is not None and lh.numel() != B:
        raise ValueError(f"seq_lens_host must hold {B} lengths")
    opts = _options(num_ctas, flags, wait_timeout_ns, split_events, _dtype_code(q, dtype), kv, k_scale, v_scale, 1)
    mask = (_ptr(tree_mask), stride, _ptr(tree_lens), _ptr(seq_lens), _ptr(lh), B, T, hq, hkv, d)
    tail = (float(scale), _ptr(out), None if lse is False else _ptr(lse), _ptr(workspace),
            workspace.numel() * workspace.element_size(), ctypes.byref(opts))
    return dev, mask, tail, out, (None if lse is False else lse), (lh, opts, workspace)


def fd_tree_decode(q, k, v, seq_lens=None, tree_mask=None, tree_lens=None, seq_lens_host=None, scale=None, out=None,
                   lse=None, workspace=None, num_ctas=0, flags=0, wait_timeout_ns=0, split_events=None, stream=None,
                   check=True, dtype=None, kv_dtype=None, k_scale=1.0, v_scale=1.0):
    """Attention of a drafted tree over a contiguous cache (see fd_tree_decode in include/fd.h).

    q [B, T, Hq, D]; k/v [B, S, Hkv, D] with the T nodes as the last positions
    of every request; tree_mask int64/uint64 words [B, T, ceil(T / 64)], or
    [T, ceil(T / 64)] for all requests (bit j of row i: node i sees node j;
    None: a causal chain); tree_lens int32 [B] (None: T nodes each).  The other
    arguments are fd_decode's.  Returns (out fp32 [B, T, Hq, D], lse [B, T, Hq])."""
    dev, mask, tail, out, lse_out, keep = _tree_args(
        q, k, v, tree_mask, tree_lens, seq_lens, seq_lens_host, scale, out, lse, workspace, num_ctas, flags,
        wait_timeout_ns, split_events, dtype, kv_dtype, k_scale, v_scale, None)
    st = _launch(dev, _lib.fd_tree_decode, _ptr(q), _ptr(k), _ptr(v), *mask, k.shape[1], *tail,
                 _stream_ptr(stream, dev))
    if check and st != FD_OK:
        raise FdError(st, "fd_tree_decode")
    return out, lse_out


def fd_tree_decode_paged(q, k_pages, v_pages, block_table, seq_lens, tree_mask=None, tree_lens=None,
                         seq_lens_host=None, scale=None, out=None, lse=None, workspace=None, num_ctas=0, flags=0,
                         wait_timeout_ns=0, split_events=None, stream=None, check=True, dtype=None, kv_dtype=None,
                         k_scale=1.0, v_scale=1.0):
    """fd_tree_decode over pages [num_pages, P, Hkv, D] behind block_table int32 [B, max_blocks]."""
    if seq_lens is None or block_table is None:
        raise ValueError("a paged cache needs its block_table and seq_lens")
    dev, mask, tail, out, lse_out, keep = _tree_args(
        q, k_pages, v_pages, tree_mask, tree_lens, seq_lens, seq_lens_host, scale, out, lse, workspace, num_ctas,
        flags, wait_timeout_ns, split_events, dtype, kv_dtype, k_scale, v_scale, block_table)
    st = _launch(dev, _lib.fd_tree_decode_paged, _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                 block_table.shape[1], *mask, k_pages.shape[1], k_pages.shape[0], *tail, _stream_ptr(stream, dev))
    if check and st != FD_OK:
        raise FdError(st, "fd_tree_decode_paged")
    return out, lse_out
