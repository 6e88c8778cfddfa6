"""Long contexts: caches in 4 bits, and attention through a sliding window with
sinks: the binding of fd_cache_write4, fd_cache_read4, fd_decode4,
fd_window_decode and their paged forms (include/fd.h).

    cache = make_cache4(num_pages, kv_heads, page, head_dim)
    fd_cache_write4(k_new, v_new, slot_map, cache, k_scale=ks, v_scale=vs)
    out, lse = fd_decode4_paged(q, cache, table, seq_lens, k_scale=ks, v_scale=vs)
    out, lse = fd_window_decode_paged(q, k_pages, v_pages, table, seq_lens, window=4096, sinks=4)

Like the package's other functions these only check and marshal arguments;
tensors live on one GPU, outputs are allocated unless they are given.  A call
runs on that GPU's current stream, whatever device is current, or on the
stream given as `stream=`, one of that GPU, which then owns what the call
allocates.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import FD_ERR_INVALID_ARG, FD_OK, FdCache4, FdError, FdOptions, _kv_code, _lib, _options, fd_workspace_init
from .speculative import _BF16, _F16, _F32, _I32, _I64, _gpu, _launch, _on_stream, _ptr_of, _status, _table_of, _token_rows

__all__ = ["Cache4", "make_cache4", "fd_cache_write4", "fd_cache_read4", "fd_decode4", "fd_decode4_paged",
           "fd_window_decode", "fd_window_decode_paged", "fd_window_workspace_size", "make_window_workspace"]

_U8 = torch.uint8


class Cache4(NamedTuple):
    """A 4-bit cache (fd_cache4 in include/fd.h): pages [num_pages, Hkv, P, ..], or contiguous [B, Hkv, S, ..].

    Codes are uint8 [.., D / 2], two a byte; scales are E4M3 [.., D / 16], as
    torch.float8_e4m3fn or as uint8 codes."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def make_cache4(pages, num_kv_heads, page_size, head_dim, device="cuda") -> Cache4:
    """Allocate (with torch) a 4-bit cache of zeros: `pages` pages of page_size tokens, or `pages` requests of page_size."""
    def zeros(width, dtype):
        return torch.zeros(pages, num_kv_heads, page_size, width, dtype=_U8, device=device).view(dtype)
    return Cache4(zeros(head_dim // 2, _U8), zeros(head_dim // 16, torch.float8_e4m3fn), zeros(head_dim // 2, _U8),
                  zeros(head_dim // 16, torch.float8_e4m3fn))


def _cache(cache, d, gpu):
    """(FdCache4, (pages, Hkv, page)) of a cache of head dim d on the call's GPU."""
    kc, ks, vc, vs = cache
    if kc.dim() != 4:
        raise ValueError(f"k_codes must be [pages, Hkv, P, {d // 2}], got {list(kc.shape)}")
    lead = kc.shape[:3]
    codes, scales = (*lead, d // 2), (*lead, d // 16)
    for t, name in ((ks, "k_scales"), (vs, "v_scales")):
        if t.dtype is not torch.float8_e4m3fn and t.dtype is not _U8:
            raise ValueError(f"{name} must be float8_e4m3fn or uint8, got {t.dtype}")
    return FdCache4(_ptr_of(kc, "k_codes", _U8, codes, gpu), _ptr_of(ks, "k_scales", ks.dtype, scales, gpu),
                    _ptr_of(vc, "v_codes", _U8, codes, gpu), _ptr_of(vs, "v_scales", vs.dtype, scales, gpu)), lead


def _rows4(name, call, k, v, kn, vn, slot_map, cache, k_scale, v_scale, device_status, check, stream, write):
    """Both directions: 16-bit rows k, v [n, Hkv, D] and the slots of a 4-bit cache."""
    gpu = _gpu(slot_map, "slot_map", stream)
    ks, vs = _token_rows(k, kn, gpu), _token_rows(v, vn, gpu)
    n, h, d = shape = k.shape
    if v.shape != shape or v.dtype is not k.dtype:
        raise ValueError(f"{kn} and {vn} must have one shape and type")
    c, (pages, heads, page) = _cache(cache, d, gpu)
    if heads != h:
        raise ValueError(f"the cache has {heads} kv heads, the rows {h}")
    opts = FdOptions(0, 0, 0, None, None, 1 if k.dtype is _F16 else 0, 0, k_scale, v_scale, 1)
    slots = _ptr_of(slot_map, "slot_map", _I64, (n,), gpu)
    status = _status(device_status, gpu)
    if write:
        st = _launch(gpu, call, k.data_ptr(), v.data_ptr(), ks, vs, slots, n, h, d, c, page, pages * page, opts, status)
    else:
        st = _launch(gpu, call, slots, n, h, d, c, page, pages * page, k.data_ptr(), v.data_ptr(), ks, vs, opts, status)
    if check and st != FD_OK:
        raise FdError(st, name)


@_on_stream
def fd_cache_write4(k_new, v_new, slot_map, cache, k_scale=1.0, v_scale=1.0, device_status=None, check=True, *,
                    stream=None):
    """Quantise new K/V rows into a 4-bit cache's slots (see fd_cache_write4 in include/fd.h).

    k_new, v_new bf16 or fp16 [n, Hkv, D], any token stride that is a multiple
    of 8; slot_map int64 [n] (negative: skip); cache a Cache4; k_scale and
    v_scale the tensors' scales."""
    _rows4("fd_cache_write4", _lib.fd_cache_write4, k_new, v_new, "k_new", "v_new", slot_map, cache, k_scale, v_scale,
           device_status, check, stream, True)


@_on_stream
def fd_cache_read4(slot_map, cache, dtype=_BF16, k_out=None, v_out=None, k_scale=1.0, v_scale=1.0, device_status=None,
                   check=True, *, stream=None):
    """Rows of a 4-bit cache's slots as 16-bit rows (see fd_cache_read4 in include/fd.h).

    Returns (k, v) [n, Hkv, D]: k_out and v_out where given (any token stride
    that is a multiple of 8), else new tensors of `dtype` (bf16 or fp16). The
    rows of negative slots keep what they hold; in new tensors they are 0."""
    if k_out is None or v_out is None:
        codes = cache[0]
        shape = (slot_map.shape[0], codes.shape[1], 2 * codes.shape[3])
        k_out = torch.zeros(shape, dtype=dtype, device=codes.device) if k_out is None else k_out
        v_out = torch.zeros(shape, dtype=dtype, device=codes.device) if v_out is None else v_out
    _rows4("fd_cache_read4", _lib.fd_cache_read4, k_out, v_out, "k_out", "v_out", slot_map, cache, k_scale, v_scale,
           device_status, check, stream, False)
    return k_out, v_out


def fd_window_workspace_size(batch, num_q_heads, num_kv_heads, head_dim=128, q_len=1) -> int:
    return int(_lib.fd_window_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, q_len))


def make_window_workspace(batch, num_q_heads, num_kv_heads, head_dim=128, device="cuda", q_len=1) -> torch.Tensor:
    """Allocate (with torch) and initialise a workspace of fd_window_decode and fd_decode4 for this shape."""
    n = fd_window_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, q_len)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_window_workspace_size")
    ws = torch.empty(n, dtype=_U8, device=device)
    with torch.cuda.device(ws.device):
        fd_workspace_init(ws)
    return ws


def _attend(name, call, q, cache, pages, page, hkv, block_table, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
            workspace, num_ctas, split_events, check, kv, k_scale, v_scale, gpu):
    """Any cache: checks, outputs, and the call `name`; `cache`: its arguments in that call."""
    dt = q.dtype
    if q.dim() not in (3, 4) or not q.is_contiguous() or (dt is not _BF16 and dt is not _F16):
        raise ValueError("q must be a contiguous bf16 or fp16 tensor [B, Hq, D] or [B, q_len, Hq, D]")
    shape = q.shape
    B, T, hq, d = shape if len(shape) == 4 else (shape[0], 1, *shape[1:])
    per_request = (B,)
    layout, cap = (), (page,)
    if block_table is not None:
        layout, cap = _table_of(block_table, B, gpu), (page, pages)
    elif pages != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {pages}")
    if out is None:
        out = torch.empty(shape, dtype=_F32, device=q.device)
    if lse is None:
        lse = torch.empty(shape[:-1], dtype=_F32, device=q.device)
    elif lse is False:
        lse = None
    if workspace is None:
        workspace = make_window_workspace(B, hq, hkv, d, q.device, T)
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{gpu}")
    host = None
    if seq_lens_host is not None:
        host = seq_lens_host.to(_I32).contiguous().cpu()
        if host.numel() != B:
            raise ValueError(f"seq_lens_host must hold {B} lengths")
    opts = _options(num_ctas, 0, 0, split_events, 1 if dt is _F16 else 0, kv, k_scale, v_scale, T)
    st = _launch(gpu, call, q.data_ptr(), *cache, *layout,
                 None if seq_lens is None else _ptr_of(seq_lens, "seq_lens", _I32, per_request, gpu),
                 None if host is None else host.data_ptr(), B, hq, hkv, d, *cap, window, sinks,
                 1.0 / math.sqrt(d) if scale is None else scale, _ptr_of(out, "out", _F32, shape, gpu),
                 None if lse is None else _ptr_of(lse, "lse", _F32, shape[:-1], gpu), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), opts)
    if check and st != FD_OK:
        raise FdError(st, name)
    return out, lse


def _window(name, call, q, k, v, block_table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace, num_ctas,
            split_events, check, kv_dtype, k_scale, v_scale, stream):
    gpu = _gpu(q, "q", stream)
    kv = _kv_code(k, v, kv_dtype)
    if k.dim() != 4 or k.shape != v.shape or k.get_device() != gpu or v.get_device() != gpu or k.shape[3] != q.shape[-1]:
        raise ValueError(f"k and v must have one 4-d shape with head_dim {q.shape[-1]} on cuda:{gpu}")
    if kv == 0 and (k.dtype is not q.dtype or v.dtype is not q.dtype):
        raise TypeError("a 16-bit cache must be of q's type")
    pages, page, hkv, _ = k.shape
    return _attend(name, call, q, (k.data_ptr(), v.data_ptr()), pages, page, hkv, block_table, seq_lens, window, sinks,
                   seq_lens_host, scale, out, lse, workspace, num_ctas, split_events, check, kv, k_scale, v_scale, gpu)


@_on_stream
def fd_window_decode(q, k, v, seq_lens, window, sinks=0, seq_lens_host=None, scale=None, out=None, lse=None,
                     workspace=None, num_ctas=0, split_events=None, check=True, kv_dtype=None, k_scale=1.0,
                     v_scale=1.0, *, stream=None):
    """Decode attention to the last `window` and the first `sinks` positions of a
    contiguous cache (see fd_window_decode in include/fd.h).

    q [B, Hq, D] or [B, q_len, Hq, D]; k/v [B, S, Hkv, D] of q's type or FP8
    (float8 tensors, or uint8 codes with kv_dtype 'e4m3' / 'e5m2'); seq_lens
    int32 [B] or None (every request has S tokens).  Returns (out fp32 of q's
    shape, lse); lse=False skips the LSE."""
    return _window("fd_window_decode", _lib.fd_window_decode, q, k, v, None, seq_lens, window, sinks, seq_lens_host, scale, out,
                   lse, workspace, num_ctas, split_events, check, kv_dtype, k_scale, v_scale, stream)


@_on_stream
def fd_window_decode_paged(q, k_pages, v_pages, block_table, seq_lens, window, sinks=0, seq_lens_host=None, scale=None,
                           out=None, lse=None, workspace=None, num_ctas=0, split_events=None, check=True, kv_dtype=None,
                           k_scale=1.0, v_scale=1.0, *, stream=None):
    """fd_window_decode over pages [num_pages, P, Hkv, D] behind block_table int32
    [B, max_blocks]; entries of pages without a visible position may hold anything."""
    if seq_lens is None or block_table is None:
        raise ValueError("a paged cache needs its block_table and seq_lens")
    return _window("fd_window_decode_paged", _lib.fd_window_decode_paged, q, k_pages, v_pages, block_table, seq_lens, window,
                   sinks, seq_lens_host, scale, out, lse, workspace, num_ctas, split_events, check, kv_dtype, k_scale,
                   v_scale, stream)


def _decode4(name, call, q, cache, block_table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace, num_ctas,
             split_events, check, k_scale, v_scale, stream):
    gpu = _gpu(q, "q", stream)
    c, (pages, hkv, page) = _cache(cache, q.shape[-1], gpu)
    return _attend(name, call, q, (c,), pages, page, hkv, block_table, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
                   workspace, num_ctas, split_events, check, 0, k_scale, v_scale, gpu)


@_on_stream
def fd_decode4(q, cache, seq_lens=None, window=0, sinks=0, seq_lens_host=None, scale=None, out=None, lse=None,
               workspace=None, num_ctas=0, split_events=None, check=True, k_scale=1.0, v_scale=1.0, *, stream=None):
    """Decode attention over a contiguous 4-bit cache, a Cache4 of [B, Hkv, S, ..]
    (see fd_decode4 in include/fd.h); window 0: all positions.  The other
    arguments are fd_window_decode's."""
    return _decode4("fd_decode4", _lib.fd_decode4, q, cache, None, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
                    workspace, num_ctas, split_events, check, k_scale, v_scale, stream)


@_on_stream
def fd_decode4_paged(q, cache, block_table, seq_lens, window=0, sinks=0, seq_lens_host=None, scale=None, out=None,
                     lse=None, workspace=None, num_ctas=0, split_events=None, check=True, k_scale=1.0, v_scale=1.0, *,
                     stream=None):
    """fd_decode4 over a Cache4 of pages [num_pages, Hkv, P, ..] behind block_table int32 [B, max_blocks]."""
    if seq_lens is None or block_table is None:
        raise ValueError("a paged cache needs its block_table and seq_lens")
    return _decode4("fd_decode4_paged", _lib.fd_decode4_paged, q, cache, block_table, seq_lens, window, sinks, seq_lens_host,
                    scale, out, lse, workspace, num_ctas, split_events, check, k_scale, v_scale, stream)
