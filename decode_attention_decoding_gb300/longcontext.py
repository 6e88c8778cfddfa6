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
allocates.  Short calls take less time on the GPU than here, so the checks are
kept to a few attribute reads a tensor; a program keeps a workspace
(make_window_workspace) and gives it to its calls, which otherwise allocate and
zero one each.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch

from . import FD_ERR_INVALID_ARG, FD_OK, FdCache4, FdError, FdOptions, _kv_code, _lib, _options, fd_workspace_init
from .speculative import _BF16, _F16, _F32, _I32, _I64, _gpu, _on_stream, _ptr_of, _status, _table_of, _token_rows

__all__ = ["Cache4", "make_cache4", "fd_cache_write4", "fd_cache_read4", "fd_decode4", "fd_decode4_paged",
           "fd_window_decode", "fd_window_decode_paged", "fd_window_workspace_size", "make_window_workspace"]

_U8 = torch.uint8
_SCALES = (torch.float8_e4m3fn, torch.uint8)
_INT = 1 << 31


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


_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _call(gpu, f, *args):
    """Call f with the GPU's current stream as its last argument and the GPU current (kernels launch on the current one)."""
    if _current_device() == gpu:
        return f(*args, _raw_stream(gpu))
    with torch.cuda.device(gpu):
        return f(*args, _raw_stream(gpu))


def _held(num_ctas, *scales):
    """Refuses what the options' C types do not hold: ctypes would pass num_ctas's low 32 bits, and a scale below fp32's
    least number as 0, which stands for 1."""
    if not -_INT <= num_ctas < _INT:
        raise ValueError(f"num_ctas must be below 2^31 in magnitude, got {num_ctas}")
    for x in scales:
        if x != 0 and ctypes.c_float(x).value == 0:
            raise ValueError(f"a scale of {x} is 0 in fp32")


@functools.lru_cache(maxsize=256)
def _opts(num_ctas, dtype, kv, k_scale, v_scale, q_len):
    """The options of these values; the library only reads them."""
    _held(num_ctas, k_scale, v_scale)
    return FdOptions(num_ctas, 0, 0, None, None, dtype, kv, k_scale, v_scale, q_len)


def _cache(cache, d, gpu):
    """(FdCache4, pages, Hkv, page) of a cache of head dim d on the call's GPU."""
    kc, ks, vc, vs = cache
    codes, scales = kc.shape, ks.shape
    ok = (kc.dtype is _U8 and vc.dtype is _U8 and len(codes) == 4 and 2 * codes[3] == d and vc.shape == codes and kc.get_device() == gpu
          and vc.get_device() == gpu and kc.is_contiguous() and vc.is_contiguous())
    if not ok:
        raise ValueError(f"k_codes and v_codes must be contiguous uint8 [pages, Hkv, P, {d // 2}] on cuda:{gpu}, got {kc.dtype} "
                         f"{list(kc.shape)} on {kc.device} and {vc.dtype} {list(vc.shape)} on {vc.device}")
    pages, hkv, page, _ = codes
    ok = (ks.dtype in _SCALES and vs.dtype in _SCALES and scales == (pages, hkv, page, d // 16) and vs.shape == scales
          and ks.get_device() == gpu and vs.get_device() == gpu and ks.is_contiguous() and vs.is_contiguous())
    if not ok:
        raise ValueError(f"k_scales and v_scales must be contiguous float8_e4m3fn or uint8 {[pages, hkv, page, d // 16]} on cuda:{gpu}, got "
                         f"{ks.dtype} {list(ks.shape)} on {ks.device} and {vs.dtype} {list(vs.shape)} on {vs.device}")
    return FdCache4(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr()), pages, hkv, page


def _rows4(name, call, k, v, kn, vn, slot_map, cache, k_scale, v_scale, device_status, check, stream, write):
    """Both directions: 16-bit rows k, v [n, Hkv, D] and the slots of a 4-bit cache."""
    gpu = _gpu(slot_map, "slot_map", stream)
    ks, vs = _token_rows(k, kn, gpu), _token_rows(v, vn, gpu)
    n, h, d = shape = k.shape
    if v.shape != shape or v.dtype is not k.dtype:
        raise ValueError(f"{kn} and {vn} must have one shape and type")
    c, pages, heads, page = _cache(cache, d, gpu)
    if heads != h:
        raise ValueError(f"the cache has {heads} kv heads, the rows {h}")
    opts = _opts(0, 1 if k.dtype is _F16 else 0, 0, float(k_scale), float(v_scale), 1)
    slots = _ptr_of(slot_map, "slot_map", _I64, (n,), gpu)
    status = None if device_status is None else _status(device_status, gpu)
    if write:
        st = _call(gpu, call, k.data_ptr(), v.data_ptr(), ks, vs, slots, n, h, d, c, page, pages * page, opts, status)
    else:
        st = _call(gpu, call, slots, n, h, d, c, page, pages * page, k.data_ptr(), v.data_ptr(), ks, vs, opts, status)
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
    shape = (batch, num_q_heads, num_kv_heads, head_dim, q_len)
    if not all(0 <= x < _INT for x in shape):   # ctypes would pass their low 32 bits
        return 0
    return int(_lib.fd_window_workspace_size(*shape))


def make_window_workspace(batch, num_q_heads, num_kv_heads, head_dim=128, device="cuda", q_len=1) -> torch.Tensor:
    """Allocate (with torch) and initialise a workspace of fd_window_decode and fd_decode4 for this shape."""
    n = fd_window_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, q_len)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_window_workspace_size")
    ws = torch.empty(n, dtype=_U8, device=device)
    with torch.cuda.device(ws.device):
        fd_workspace_init(ws)
    return ws


def _attend(name, call, q, gpu, cache, pages, page, hkv, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
            workspace, num_ctas, split_events, check, kv, k_scale, v_scale):
    """Any cache: checks, outputs, and the call `name`; `cache`: its arguments in that call."""
    if not (-_INT <= window < _INT and -_INT <= sinks < _INT):   # ctypes would pass their low 32 bits
        raise ValueError(f"window and sinks must be below 2^31 in magnitude, got {window} and {sinks}")
    shape, dt = q.shape, q.dtype
    if len(shape) == 4:
        B, T, hq, d = shape
    elif len(shape) == 3:
        (B, hq, d), T = shape, 1
    else:
        raise ValueError(f"q must be [B, Hq, D] or [B, q_len, Hq, D], got {list(shape)}")
    if (dt is not _BF16 and dt is not _F16) or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 or fp16 tensor")
    if table is not None:
        layout = (*_table_of(table, B, gpu),)
        cap = (page, pages)
    elif pages != B:
        raise ValueError(f"a contiguous cache must hold {B} requests, got {pages}")
    else:
        layout, cap = (), (page,)
    if out is None:
        out = torch.empty(shape, dtype=_F32, device=q.device)
    else:
        _ptr_of(out, "out", _F32, shape, gpu)
    if lse is None:
        lse = torch.empty(shape[:-1], dtype=_F32, device=q.device)
    elif lse is False:
        lse = None
    else:
        _ptr_of(lse, "lse", _F32, shape[:-1], gpu)
    if workspace is None:
        workspace = make_window_workspace(B, hq, hkv, d, q.device, T)
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{gpu}")
    host = None
    if seq_lens_host is not None:
        host = seq_lens_host.to(_I32).contiguous().cpu()
        if host.numel() != B:
            raise ValueError(f"seq_lens_host must hold {B} lengths")
    f16 = 1 if dt is _F16 else 0
    if split_events is None:
        opts = _opts(num_ctas, f16, kv, float(k_scale), float(v_scale), T)
    else:
        _held(num_ctas, k_scale, v_scale)
        opts = _options(num_ctas, 0, 0, split_events, f16, kv, k_scale, v_scale, T)
    st = _call(gpu, call, q.data_ptr(), *cache, *layout, None if seq_lens is None else _ptr_of(seq_lens, "seq_lens", _I32, (B,), gpu),
               None if host is None else host.data_ptr(), B, hq, hkv, d, *cap, window, sinks,
               1.0 / math.sqrt(d) if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
               workspace.data_ptr(), workspace.nbytes, opts)
    if check and st != FD_OK:
        raise FdError(st, name)
    return out, lse


def _window(name, call, q, k, v, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace, num_ctas,
            split_events, check, kv_dtype, k_scale, v_scale, stream):
    gpu = q.get_device()
    if gpu < 0 or stream is not None:
        _gpu(q, "q", stream)
        with torch.cuda.stream(stream):
            return _window(name, call, q, k, v, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace,
                           num_ctas, split_events, check, kv_dtype, k_scale, v_scale, None)
    shape, dt = k.shape, k.dtype
    if (len(shape) != 4 or v.shape != shape or shape[3] != q.shape[-1] or k.get_device() != gpu or v.get_device() != gpu
            or not k.is_contiguous() or not v.is_contiguous()):
        raise ValueError(f"k and v must be contiguous, of one 4-d shape with head_dim {q.shape[-1]}, on cuda:{gpu}")
    kv = 0
    if kv_dtype is not None or dt is not q.dtype or v.dtype is not dt:
        kv = _kv_code(k, v, kv_dtype)
        if kv == 0:
            raise TypeError("a 16-bit cache must be of q's type")
    pages, page, hkv, _ = shape
    return _attend(name, call, q, gpu, (k.data_ptr(), v.data_ptr()), pages, page, hkv, table, seq_lens, window, sinks, seq_lens_host,
                   scale, out, lse, workspace, num_ctas, split_events, check, kv, k_scale, v_scale)


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


def _decode4(name, call, q, cache, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace, num_ctas,
             split_events, check, k_scale, v_scale, stream):
    gpu = q.get_device()
    if gpu < 0 or stream is not None:
        _gpu(q, "q", stream)
        with torch.cuda.stream(stream):
            return _decode4(name, call, q, cache, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse, workspace,
                            num_ctas, split_events, check, k_scale, v_scale, None)
    c, pages, hkv, page = _cache(cache, q.shape[-1], gpu)
    return _attend(name, call, q, gpu, (c,), pages, page, hkv, table, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
                   workspace, num_ctas, split_events, check, 0, k_scale, v_scale)


def fd_decode4(q, cache, seq_lens=None, window=0, sinks=0, seq_lens_host=None, scale=None, out=None, lse=None,
               workspace=None, num_ctas=0, split_events=None, check=True, k_scale=1.0, v_scale=1.0, *, stream=None):
    """Decode attention over a contiguous 4-bit cache, a Cache4 of [B, Hkv, S, ..]
    (see fd_decode4 in include/fd.h); window 0: all positions.  The other
    arguments are fd_window_decode's."""
    return _decode4("fd_decode4", _lib.fd_decode4, q, cache, None, seq_lens, window, sinks, seq_lens_host, scale, out, lse,
                    workspace, num_ctas, split_events, check, k_scale, v_scale, stream)


def fd_decode4_paged(q, cache, block_table, seq_lens, window=0, sinks=0, seq_lens_host=None, scale=None, out=None,
                     lse=None, workspace=None, num_ctas=0, split_events=None, check=True, k_scale=1.0, v_scale=1.0, *,
                     stream=None):
    """fd_decode4 over a Cache4 of pages [num_pages, Hkv, P, ..] behind block_table int32 [B, max_blocks]."""
    if seq_lens is None or block_table is None:
        raise ValueError("a paged cache needs its block_table and seq_lens")
    return _decode4("fd_decode4_paged", _lib.fd_decode4_paged, q, cache, block_table, seq_lens, window, sinks, seq_lens_host,
                    scale, out, lse, workspace, num_ctas, split_events, check, k_scale, v_scale, stream)
