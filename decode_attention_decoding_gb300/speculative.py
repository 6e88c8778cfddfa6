"""A step of speculative decoding over a KV cache: the binding of
fd_build_tables, fd_cache_write, fd_tree_decode, fd_tree_decode_paged and
fd_cache_compact (include/fd.h).

    tables = fd_build_tables(lens, new_lens, table, free, free_count, page, num_pages, max_tokens)
    fd_cache_write(k_new, v_new, tables.slot_map, k_pages, v_pages)
    out, lse = fd_tree_decode_paged(q, k_pages, v_pages, table, tables.seq_lens, mask)
    lens = fd_cache_compact(k_pages, v_pages, tables.seq_lens, accepted, accept_lens, tree_len, block_table=table)

Like the package's other functions these only check and marshal arguments;
tensors live on one GPU, outputs are allocated unless they are given.  A call
runs on that GPU's current stream, whatever device is current, or on the
stream given as `stream=`, one of that GPU, which then owns what the call
allocates.  These
calls take a few microseconds on the GPU, so the checks are kept to a few
attribute reads a tensor.
"""
from __future__ import annotations

import functools
import math
from typing import NamedTuple

import torch

from . import (FD_ERR_INVALID_ARG, FD_OK, FdError, FdOptions, _dtype_code, _kv_code, _lib, _options,
               fd_workspace_init)

__all__ = ["fd_build_tables", "fd_cache_write", "fd_cache_compact", "fd_tree_workspace_size", "make_tree_workspace",
           "fd_tree_decode", "fd_tree_decode_paged", "Tables", "FD_DEVICE_STATUS_BAD_LENGTH",
           "FD_DEVICE_STATUS_NO_PAGES", "FD_DEVICE_STATUS_BAD_SLOT"]

FD_DEVICE_STATUS_BAD_LENGTH, FD_DEVICE_STATUS_NO_PAGES, FD_DEVICE_STATUS_BAD_SLOT = 0x2, 0x4, 0x8

_I32, _F32, _I64, _BF16, _F16 = torch.int32, torch.float32, torch.int64, torch.bfloat16, torch.float16


class Tables(NamedTuple):
    """What fd_build_tables gives back."""
    block_table: torch.Tensor   # [B, max_blocks] int32, the caller's, updated
    slot_map: torch.Tensor      # [max_tokens] int64
    cu_new_lens: torch.Tensor   # [B + 1] int32
    seq_lens: torch.Tensor      # [B] int32, with the new tokens
    held_pages: torch.Tensor    # [B] int32
    free_count: torch.Tensor    # [1] int32


def _gpu(t, name, stream):
    """Index of the GPU that t, and the stream if one is given, is on."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, {name} on cuda:{index}")
    return index


def _ptr_of(t, name, dtype, shape, gpu):
    """Address of a contiguous tensor of this type and shape on the call's GPU."""
    if t.dtype is not dtype or t.get_device() != gpu or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{gpu}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _table_of(t, rows, gpu):
    """(address, columns) of a block table [rows, max_blocks]."""
    if t.dim() != 2:
        raise ValueError(f"block_table must be [{rows}, max_blocks], got {list(t.shape)}")
    return _ptr_of(t, "block_table", _I32, (rows, t.shape[1]), gpu), t.shape[1]


def _status(t, gpu):
    if t is None:
        return None
    if t.dtype not in (torch.int32, torch.uint32) or t.get_device() != gpu or t.numel() != 1:
        raise ValueError("device_status must be one int32 or uint32 on the call's device")
    return t.data_ptr()


def _launch(gpu, f, *args):
    """Call f with the GPU's current stream as its last argument and the GPU current (kernels launch on the current one)."""
    s = torch._C._cuda_getCurrentRawStream(gpu)   # torch.cuda.current_stream(gpu).cuda_stream without the object: 0.1 us, not 1.1
    if torch.cuda.current_device() == gpu:
        return f(*args, s)
    with torch.cuda.device(gpu):
        return f(*args, s)


def _on_stream(f):
    """f(.., stream=s) as f(..) with s current, so that what f allocates belongs to s and is initialised on it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, stream=stream, **kw)
    return call


@_on_stream
def fd_build_tables(seq_lens, new_lens, block_table, free_pages, free_count, page_size, num_pages, max_tokens,
                    held_pages=None, slot_map=None, device_status=None, check=True, *, stream=None):
    """Give requests pages and slots for their new tokens (see fd_build_tables in include/fd.h).

    seq_lens, new_lens and held_pages int32 [B]; block_table int32 [B,
    max_blocks], updated in place; free_pages int32 [n], a stack whose first
    free_count (int32 [1]) entries are free; max_tokens the length of the slot
    map (entries behind the last token are -1).  Returns a Tables."""
    gpu = _gpu(block_table, "block_table", stream)
    B = seq_lens.shape[0]
    per_request, n = (B,), int(max_tokens)
    table, blocks = _table_of(block_table, B, gpu)
    dev = block_table.device
    if slot_map is None:
        slot_map = torch.empty(n, dtype=_I64, device=dev)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be 1-d")
    cu, lens, held, left = torch.split_with_sizes(torch.empty(3 * B + 2, dtype=_I32, device=dev), (B + 1, B, B, 1))
    st = _launch(gpu, _lib.fd_build_tables, _ptr_of(seq_lens, "seq_lens", _I32, per_request, gpu),
                 _ptr_of(new_lens, "new_lens", _I32, per_request, gpu),
                 None if held_pages is None else _ptr_of(held_pages, "held_pages", _I32, per_request, gpu),
                 _ptr_of(free_pages, "free_pages", _I32, free_pages.shape, gpu),
                 _ptr_of(free_count, "free_count", _I32, (1,), gpu), free_pages.shape[0], B, int(page_size),
                 int(num_pages), blocks, n, table, _ptr_of(slot_map, "slot_map", _I64, (n,), gpu), cu.data_ptr(),
                 lens.data_ptr(), held.data_ptr(), left.data_ptr(), _status(device_status, gpu))
    if check and st != FD_OK:
        raise FdError(st, "fd_build_tables")
    return Tables(block_table, slot_map, cu, lens, held, left)


def _token_rows(t, name, gpu):
    """Check new K or V rows [n, Hkv, D], dense inside a token's row; their stride in elements."""
    if (t.dtype is not _BF16 and t.dtype is not _F16) or t.dim() != 3 or t.get_device() != gpu:
        raise ValueError(f"{name} must be a bf16 or fp16 tensor [n, Hkv, D] on cuda:{gpu}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    token, head, element = t.stride()
    if element != 1 or (head != t.shape[2] and t.shape[1] > 1):
        raise ValueError(f"{name}: a token's heads must be dense (only the token stride is free)")
    return token


@_on_stream
def fd_cache_write(k_new, v_new, slot_map, k_cache, v_cache, kv_dtype=None, k_scale=1.0, v_scale=1.0,
                   device_status=None, check=True, *, stream=None):
    """Write new K/V rows into the cache's slots (see fd_cache_write in include/fd.h).

    k_new, v_new bf16 or fp16 [n, Hkv, D], any token stride that is a multiple
    of 8; slot_map int64 [n] (negative: skip); k_cache, v_cache [..., Hkv, D]
    (pages [num_pages, P, Hkv, D], a contiguous cache [B, S, Hkv, D], or flat
    slots) of the same type, or FP8: float8 tensors, or uint8 codes with
    kv_dtype 'e4m3' / 'e5m2', quantised by k_scale / v_scale."""
    gpu = _gpu(k_cache, "k_cache", stream)
    ks, vs = _token_rows(k_new, "k_new", gpu), _token_rows(v_new, "v_new", gpu)
    kv = _kv_code(k_cache, v_cache, kv_dtype)
    n, h, d = shape = k_new.shape
    if v_new.shape != shape or v_new.dtype is not k_new.dtype:
        raise ValueError("k_new and v_new must have one shape and type")
    if k_cache.shape != v_cache.shape or v_cache.get_device() != gpu or k_cache.dim() < 3 or k_cache.shape[-2:] != (h, d):
        raise ValueError(f"k_cache and v_cache must have one shape [..., {h}, {d}] on one device")
    if kv == 0 and (k_cache.dtype is not k_new.dtype or v_cache.dtype is not k_new.dtype):
        raise TypeError("a 16-bit cache must be of the new rows' type")
    opts = FdOptions(0, 0, 0, None, None, 1 if k_new.dtype is _F16 else 0, kv, k_scale, v_scale, 1)
    st = _launch(gpu, _lib.fd_cache_write, k_new.data_ptr(), v_new.data_ptr(), ks, vs,
                 _ptr_of(slot_map, "slot_map", _I64, (n,), gpu), n, h, d, k_cache.data_ptr(), v_cache.data_ptr(),
                 k_cache.numel() // (h * d) if h * d else 0, opts, _status(device_status, gpu))
    if check and st != FD_OK:
        raise FdError(st, "fd_cache_write")


@_on_stream
def fd_cache_compact(k_cache, v_cache, seq_lens, accepted, accept_lens, tree_len, block_table=None, tree_lens=None,
                     seq_lens_out=None, device_status=None, check=True, *, stream=None):
    """Move the accepted path's rows to the front of the drafted tail, in place
    (see fd_cache_compact in include/fd.h).

    k_cache, v_cache [B, S, Hkv, D], or pages [num_pages, P, Hkv, D] with
    block_table int32 [B, max_blocks], of any type a cache has; seq_lens int32
    [B] with the drafted tokens; accepted int32 [B, max_accept], ascending node
    indices; accept_lens int32 [B]; tree_lens int32 [B] or None (tree_len for
    every request).  Returns the new lengths int32 [B]."""
    gpu = _gpu(k_cache, "k_cache", stream)
    B = seq_lens.shape[0]
    per_request = (B,)
    size = k_cache.element_size()
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_contiguous() or t.dim() != 4 or t.get_device() != gpu or size > 2:
            raise ValueError(f"{name} must be a contiguous 4-d tensor of 16-bit or FP8 elements on cuda:{gpu}")
    if k_cache.shape != v_cache.shape or size != v_cache.element_size():
        raise ValueError("k_cache and v_cache must have one shape and type")
    if accepted.dim() != 2:
        raise ValueError(f"accepted must be [{B}, max_accept], got {list(accepted.shape)}")
    pages, page, h, d = k_cache.shape
    table, blocks = None, 0
    if block_table is not None:
        table, blocks = _table_of(block_table, B, gpu)
    elif pages != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {pages}")
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens)
    most = accepted.shape[1]
    opts = FdOptions(0, 0, 0, None, None, 0, 1 if size == 1 else 0, 0.0, 0.0, 1)
    st = _launch(gpu, _lib.fd_cache_compact, k_cache.data_ptr(), v_cache.data_ptr(), table, blocks, page, pages,
                 _ptr_of(seq_lens, "seq_lens", _I32, per_request, gpu),
                 None if tree_lens is None else _ptr_of(tree_lens, "tree_lens", _I32, per_request, gpu), int(tree_len),
                 _ptr_of(accepted, "accepted", _I32, (B, most), gpu),
                 _ptr_of(accept_lens, "accept_lens", _I32, per_request, gpu), most, B, h, d,
                 _ptr_of(seq_lens_out, "seq_lens_out", _I32, per_request, gpu), opts, _status(device_status, gpu))
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
    with torch.cuda.device(ws.device):
        fd_workspace_init(ws)
    return ws


def _tree(name, q, k, v, block_table, seq_lens, tree_mask, tree_lens, seq_lens_host, scale, out, lse, workspace, num_ctas,
          flags, wait_timeout_ns, split_events, check, dtype, kv_dtype, k_scale, v_scale, stream):
    """Both layouts: checks, outputs, and the call `name`."""
    gpu = _gpu(q, "q", stream)
    if q.dim() != 4 or not q.is_contiguous() or q.element_size() != 2:
        raise ValueError("q must be a contiguous bf16 or fp16 tensor [B, tree_len, Hq, D]")
    kv = _kv_code(k, v, kv_dtype)
    B, T, hq, d = shape = q.shape
    if k.dim() != 4 or k.shape != v.shape or k.get_device() != gpu or v.get_device() != gpu or k.shape[3] != d:
        raise ValueError(f"k and v must have one 4-d shape with head_dim {d} on cuda:{gpu}")
    if kv == 0 and (k.element_size() != 2 or v.element_size() != 2 or
                    (_F16 in (q.dtype, k.dtype, v.dtype) and _BF16 in (q.dtype, k.dtype, v.dtype))):
        raise TypeError("a 16-bit cache must be of q's type")
    pages, page, hkv, _ = k.shape
    per_request = (B,)
    layout = ()
    if block_table is not None:
        layout = _table_of(block_table, B, gpu)
    elif pages != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {pages}")
    stride, words, mask = 0, (T + 63) // 64, None
    if tree_mask is not None:
        if tree_mask.dtype is not _I64 and tree_mask.dtype is not torch.uint64:
            raise ValueError("tree_mask must be int64 or uint64 words")
        if tree_mask.dim() == 3:
            stride = T * words
            mask = _ptr_of(tree_mask, "tree_mask", tree_mask.dtype, (B, T, words), gpu)
        else:
            mask = _ptr_of(tree_mask, "tree_mask", tree_mask.dtype, (T, words), gpu)
    if out is None:
        out = torch.empty(shape, dtype=_F32, device=q.device)
    if lse is None:
        lse = torch.empty((B, T, hq), dtype=_F32, device=q.device)
    elif lse is False:
        lse = None
    if workspace is None:
        workspace = make_tree_workspace(B, T, hq, hkv, d, q.device)
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{gpu}")
    host = None
    if seq_lens_host is not None:
        host = seq_lens_host.to(torch.int32).contiguous().cpu()
        if host.numel() != B:
            raise ValueError(f"seq_lens_host must hold {B} lengths")
    opts = _options(num_ctas, flags, wait_timeout_ns, split_events, _dtype_code(q, dtype), kv, k_scale, v_scale, 1)
    st = _launch(gpu, getattr(_lib, name), q.data_ptr(), k.data_ptr(), v.data_ptr(), *layout, mask, stride,
                 None if tree_lens is None else _ptr_of(tree_lens, "tree_lens", _I32, per_request, gpu),
                 None if seq_lens is None else _ptr_of(seq_lens, "seq_lens", _I32, per_request, gpu),
                 None if host is None else host.data_ptr(), B, T, hq, hkv, d, page, *((pages,) if layout else ()),
                 1.0 / math.sqrt(d) if scale is None else scale, _ptr_of(out, "out", _F32, shape, gpu),
                 None if lse is None else _ptr_of(lse, "lse", _F32, (B, T, hq), gpu), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), opts)
    if check and st != FD_OK:
        raise FdError(st, name)
    return out, lse


@_on_stream
def fd_tree_decode(q, k, v, seq_lens=None, tree_mask=None, tree_lens=None, seq_lens_host=None, scale=None, out=None,
                   lse=None, workspace=None, num_ctas=0, flags=0, wait_timeout_ns=0, split_events=None, check=True,
                   dtype=None, kv_dtype=None, k_scale=1.0, v_scale=1.0, *, stream=None):
    """Attention of a drafted tree over a contiguous cache (see fd_tree_decode in include/fd.h).

    q [B, T, Hq, D]; k/v [B, S, Hkv, D] with the T nodes as the last positions
    of every request; tree_mask int64/uint64 words [B, T, ceil(T / 64)], or
    [T, ceil(T / 64)] for all requests (bit j of row i: node i sees node j;
    None: a causal chain); tree_lens int32 [B] (None: T nodes each).  The other
    arguments are fd_decode's.  Returns (out fp32 [B, T, Hq, D], lse [B, T, Hq])."""
    return _tree("fd_tree_decode", q, k, v, None, seq_lens, tree_mask, tree_lens, seq_lens_host, scale, out, lse,
                 workspace, num_ctas, flags, wait_timeout_ns, split_events, check, dtype, kv_dtype, k_scale, v_scale, stream)


@_on_stream
def fd_tree_decode_paged(q, k_pages, v_pages, block_table, seq_lens, tree_mask=None, tree_lens=None,
                         seq_lens_host=None, scale=None, out=None, lse=None, workspace=None, num_ctas=0, flags=0,
                         wait_timeout_ns=0, split_events=None, check=True, dtype=None, kv_dtype=None,
                         k_scale=1.0, v_scale=1.0, *, stream=None):
    """fd_tree_decode over pages [num_pages, P, Hkv, D] behind block_table int32 [B, max_blocks]."""
    if seq_lens is None or block_table is None:
        raise ValueError("a paged cache needs its block_table and seq_lens")
    return _tree("fd_tree_decode_paged", q, k_pages, v_pages, block_table, seq_lens, tree_mask, tree_lens,
                 seq_lens_host, scale, out, lse, workspace, num_ctas, flags, wait_timeout_ns, split_events, check,
                 dtype, kv_dtype, k_scale, v_scale, stream)
