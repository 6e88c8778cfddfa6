"""The 4-bit cache and window calls on the host: what they refuse, with fake
device addresses (no case reaches a CUDA call), workspace sizes, and the plain
forms that the GPU tests compare with."""
import contextlib
import ctypes
import types

import numpy as np
import pytest
import torch

import longcontext_util as u

A = 1 << 20   # fake, 256-byte aligned device addresses (never dereferenced)


@pytest.fixture(scope="module")
def fd():
    from decode_attention_decoding_gb300 import build
    build.build()
    import decode_attention_decoding_gb300 as fd
    return fd


def opts(fd, **kw):
    o = fd.FdOptions(0, 0, 0, None, None, 0, 0, 0.0, 0.0, 0)
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def cache4(fd, **over):
    a = dict(k_codes=A, k_scales=2 * A, v_codes=3 * A, v_scales=4 * A)
    a.update(over)
    return ctypes.byref(fd.FdCache4(**a))


def rows4(fd, write, **over):
    a = dict(k=A, v=2 * A, ks=256, vs=256, slots=3 * A, n=4, h=2, d=128, c=cache4(fd), page=16, ns=64, opts=None, st=None)
    a.update(over)
    keys = ("k", "v", "ks", "vs", "slots", "n", "h", "d", "c", "page", "ns") if write else ("slots", "n", "h", "d", "c", "page", "ns", "k", "v", "ks", "vs")
    return (fd._lib.fd_cache_write4 if write else fd._lib.fd_cache_read4)(*[a[x] for x in keys], a["opts"], a["st"], None)


@pytest.mark.parametrize("write", [True, False])
def test_rows_refusals(fd, write):
    bad = [dict(k=None), dict(v=None), dict(slots=None), dict(c=None), dict(n=-1), dict(h=0), dict(ns=-16), dict(page=0),
           dict(page=-1), dict(ns=60), dict(k=A + 8), dict(v=A + 8), dict(slots=A + 4), dict(ks=255), dict(ks=248), dict(vs=260),
           dict(st=A + 1), dict(opts=opts(fd, kv_dtype=1)), dict(opts=opts(fd, dtype=2)), dict(opts=opts(fd, k_scale=-1.0)),
           dict(opts=opts(fd, v_scale=float("nan"))), dict(opts=opts(fd, v_scale=float("inf")))]
    bad += [dict(c=cache4(fd, **{x: None})) for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    bad += [dict(c=cache4(fd, **{x: A + 8})) for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    for over in bad:
        assert rows4(fd, write, **over) == fd.FD_ERR_INVALID_ARG, over
    for over in (dict(d=0), dict(d=96), dict(d=512), dict(h=(1 << 20) + 1)):
        assert rows4(fd, write, **over) == fd.FD_ERR_UNSUPPORTED, over
    assert rows4(fd, write, n=0, k=None, slots=None) == fd.FD_OK   # nothing to move: nothing is launched


def attend(fd, four, paged, **over):
    a = dict(q=A, k=A, v=A, c=cache4(fd), table=A, blocks=8, sl=A, slh=None, B=2, hq=8, hkv=2, d=128, smax=128, page=16, pages=8,
             window=64, sinks=4, scale=0.1, o=A, lse=A, ws=A, wsb=1 << 40, opts=None)
    a.update(over)
    keys = ["q"] + (["c"] if four else ["k", "v"]) + (["table", "blocks"] if paged else []) + ["sl", "slh", "B", "hq", "hkv", "d"]
    keys += ["page", "pages"] if paged else ["smax"]
    keys += ["window", "sinks", "scale", "o", "lse", "ws", "wsb", "opts"]
    name = ("fd_decode4" if four else "fd_window_decode") + ("_paged" if paged else "")
    return getattr(fd._lib, name)(*[a[x] for x in keys], None)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("four", [False, True])
def test_attention_refusals(fd, four, paged):
    long, neg = (ctypes.c_int32 * 2)(10, 129), (ctypes.c_int32 * 2)(10, -1)
    bad = [dict(q=None), dict(o=None), dict(ws=None), dict(q=A + 8), dict(o=A + 4), dict(ws=A + 16), dict(sl=A + 2), dict(lse=A + 2),
           dict(B=-1), dict(hq=6, hkv=4), dict(hkv=0), dict(hq=0), dict(window=-1), dict(sinks=-1), dict(slh=ctypes.addressof(long)),
           dict(slh=ctypes.addressof(neg)), dict(opts=opts(fd, q_len=-1)), dict(opts=opts(fd, dtype=3)),
           dict(opts=opts(fd, kv_dtype=7)), dict(opts=opts(fd, num_ctas=161)), dict(opts=opts(fd, num_ctas=-1)),
           dict(opts=opts(fd, k_scale=float("inf")))]
    bad += [dict(table=None), dict(sl=None), dict(blocks=0), dict(page=0), dict(pages=0), dict(table=A + 2)] if paged else [dict(smax=-1)]
    if four:
        bad += [dict(c=None), dict(opts=opts(fd, kv_dtype=1))]
        bad += [dict(c=cache4(fd, **{x: v})) for x in ("k_codes", "k_scales", "v_codes", "v_scales") for v in (None, A + 8)]
    else:
        bad += [dict(k=None), dict(v=None), dict(k=A + 8), dict(window=0)]
    for over in bad:
        assert attend(fd, four, paged, **over) == fd.FD_ERR_INVALID_ARG, over
    many = [dict(d=96), dict(B=5000), dict(hq=34, hkv=2), dict(opts=opts(fd, q_len=5))]
    many += [dict(page=1 << 16, blocks=1 << 15), dict(page=1 << 16, pages=1 << 16), dict(page=1 << 16, pages=1 << 15, hkv=8),
             dict(B=4096, hkv=256, hq=256, blocks=1 << 20, page=1, window=1 << 20)] if paged else \
            [dict(smax=(1 << 31) - 1, B=2), dict(B=4096, hkv=256, hq=256, smax=1 << 16)]
    for over in many:
        assert attend(fd, four, paged, **over) == fd.FD_ERR_UNSUPPORTED, over
    assert attend(fd, four, paged, wsb=16) == fd.FD_ERR_WORKSPACE_TOO_SMALL
    assert attend(fd, four, paged, B=0) == fd.FD_OK


def test_workspace_size(fd):
    size = fd.fd_window_workspace_size
    assert size(4096, 16, 1, 256) >= 256
    for args in ((-1, 8, 8, 128, 1), (5000, 8, 8, 128, 1), (1, 8, 8, 128, 0), (1, 8, 8, 128, 17), (1, 17, 1, 128, 1), (1, 6, 4, 128, 1),
                 (1, 8, 0, 128, 1), (1, 8, 8, 96, 1)):
        assert size(*args) == 0, args
    with pytest.raises(fd.FdError):
        fd.make_window_workspace(1, 32, 1)
    # one workspace serves smaller shapes
    for small, large in (((1, 8, 8, 128, 1), (7, 8, 8, 128, 1)), ((1, 8, 8, 128, 1), (1, 8, 8, 128, 3)), ((3, 8, 2, 64, 1), (3, 8, 2, 256, 1))):
        assert size(*small) <= size(*large)


class FakeTensor:
    """Says which GPU it is on; any other use is an AttributeError."""
    shape = (1,)

    def get_device(self):
        return 0


@pytest.mark.parametrize("name,args", [("fd_cache_write4", [FakeTensor()] * 4), ("fd_decode4", [FakeTensor()] * 3),
                                       ("fd_decode4_paged", [FakeTensor()] * 4), ("fd_window_decode", [FakeTensor()] * 4 + [1]),
                                       ("fd_window_decode_paged", [FakeTensor()] * 5 + [1])])
def test_a_stream_of_another_gpu_is_refused(fd, monkeypatch, name, args):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        getattr(fd, name)(*args, stream=stream)


@pytest.mark.parametrize("window, sinks", [(2 ** 31, 0), (2 ** 32 + 5, 4), (64, 2 ** 31), (64, 2 ** 32 + 1)])
def test_windows_that_an_int_does_not_hold_are_refused(fd, window, sinks):
    """ctypes would pass their low 32 bits: another window."""
    from decode_attention_decoding_gb300 import longcontext

    def call(*a):
        raise AssertionError("called")
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2\\^31"):
        longcontext._attend("f", call, q, 0, (0, 0), 1, 16, 8, None, None, window, sinks, None, None, None, None, None, 0, None,
                            True, 0, 1.0, 1.0)


def test_cpu_tensors_are_refused(fd):
    c = u.make_case(1, 2, 1, 4, 2, 64, [5, 9], kv="e2m1")
    cache = fd.Cache4(*c["pool"])
    rows = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    slots, lens = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fd.fd_cache_write4(rows, rows, slots, cache), lambda: fd.fd_cache_read4(slots, cache),
                 lambda: fd.fd_decode4(c["q"], cache, lens), lambda: fd.fd_window_decode(c["q"], rows[None], rows[None], lens, 4)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the plain forms

def test_e2m1_rounding_by_hand():
    y = np.array([0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.2500001, 1.75, 1.7499999, 2.5, 2.5000002, 3.5, 3.4999998, 5.0, 5.0000005, 7.0, -0.25,
                  -0.75, -9.0, 0.0], dtype=np.float32)
    code = [0, 1, 2, 1, 2, 3, 4, 3, 4, 5, 6, 5, 6, 7, 7, 8, 10, 15, 0]
    assert u.round_e2m1_code(y).tolist() == code


def test_e4m3_rounding_is_torch_s_below_saturation():
    x = np.concatenate([np.linspace(0, 460, 5001), np.exp2(np.linspace(-14, 8.8, 5001))]).astype(np.float32)
    x = x[x < 464]
    ref = torch.from_numpy(x).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(u.e4m3_code(x), ref)


def test_quantised_gaussians_are_near():
    """A code is off by at most 1 of its block's 6 units (between 4 and 6), 1.07 where the scale was rounded down (2^-4 at most)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 128, generator=g).bfloat16()
    codes, s = u.quantise4(x, 0.013)
    v = u.values4(codes, s, 0.013)
    x = x.double().numpy()
    top = np.abs(x).reshape(50, 8, 16).max(-1).repeat(16, -1)
    assert (np.abs(v - x) <= top / 6 * (1 + 2.0 ** -4) * 1.001).all()
    assert (np.abs(v - x) > top / 60).any()
