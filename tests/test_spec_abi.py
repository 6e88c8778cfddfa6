"""The speculative-decoding calls on the host: what they refuse, with fake
device addresses (no case reaches a CUDA call), and the workspace size."""
import ctypes

import pytest

A = 1 << 20   # fake, 256-byte aligned device addresses (never dereferenced)
P = ctypes.c_void_p


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


def tables(fd, **over):
    a = dict(sl=A, nl=2 * A, held=None, free=3 * A, count=4 * A, max_free=8, B=2, page=16, pages=8, blocks=4, tokens=8,
             table=5 * A, slots=6 * A, cu=7 * A, lo=8 * A, ho=9 * A, fo=10 * A, st=None)
    a.update(over)
    return fd._lib.fd_build_tables(*[a[k] for k in ("sl", "nl", "held", "free", "count", "max_free", "B", "page", "pages",
                                                    "blocks", "tokens", "table", "slots", "cu", "lo", "ho", "fo", "st")], None)


def test_build_tables_refusals(fd):
    bad = [dict(sl=None), dict(nl=None), dict(free=None), dict(count=None), dict(table=None), dict(slots=None),
           dict(cu=None), dict(lo=None), dict(ho=None), dict(fo=None), dict(B=-1), dict(page=0), dict(page=-16),
           dict(pages=0), dict(blocks=0), dict(tokens=-1), dict(max_free=-1), dict(sl=A + 2), dict(slots=6 * A + 4),
           dict(held=A + 1), dict(st=A + 2),
           dict(lo=A), dict(lo=A + 4), dict(ho=2 * A), dict(held=11 * A, ho=11 * A), dict(fo=4 * A), dict(cu=8 * A),
           dict(table=3 * A + 16), dict(slots=5 * A)]
    for over in bad:
        assert tables(fd, **over) == fd.FD_ERR_INVALID_ARG, over
    for over in (dict(B=5000), dict(page=1 << 20, blocks=1 << 11), dict(B=4096, blocks=1 << 20, page=1)):
        over = dict(dict(sl=A, nl=2 * A), **over)
        assert tables(fd, **over) == fd.FD_ERR_UNSUPPORTED, over


def write(fd, **over):
    a = dict(k=A, v=2 * A, ks=256, vs=256, slots=3 * A, n=4, h=2, d=128, kc=4 * A, vc=5 * A, ns=64, opts=None, st=None)
    a.update(over)
    return fd._lib.fd_cache_write(*[a[k] for k in ("k", "v", "ks", "vs", "slots", "n", "h", "d", "kc", "vc", "ns", "opts", "st")], None)


def test_cache_write_refusals(fd):
    bad = [dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(n=-1), dict(h=0),
           dict(ns=-1), dict(k=A + 8), dict(kc=A + 8), dict(slots=A + 4), dict(ks=255), dict(ks=248), dict(vs=260),
           dict(st=A + 1), dict(opts=opts(fd, kv_dtype=3)), dict(opts=opts(fd, dtype=2)),
           dict(opts=opts(fd, kv_dtype=1, k_scale=-1.0)), dict(opts=opts(fd, kv_dtype=1, v_scale=float("nan"))),
           dict(opts=opts(fd, kv_dtype=1, v_scale=float("inf")))]
    for over in bad:
        assert write(fd, **over) == fd.FD_ERR_INVALID_ARG, over
    for d in (0, 32, 96, 192, 512):
        assert write(fd, d=d) == fd.FD_ERR_UNSUPPORTED
    assert write(fd, n=0, k=None, slots=None) == fd.FD_OK   # nothing to write: nothing is launched


def compact(fd, **over):
    a = dict(k=A, v=2 * A, table=None, blocks=0, page=64, pages=0, sl=3 * A, tl=None, T=8, acc=4 * A, al=5 * A, ma=4,
             B=2, h=2, d=128, out=6 * A, opts=None, st=None)
    a.update(over)
    return fd._lib.fd_cache_compact(*[a[k] for k in ("k", "v", "table", "blocks", "page", "pages", "sl", "tl", "T", "acc",
                                                     "al", "ma", "B", "h", "d", "out", "opts", "st")], None)


def test_cache_compact_refusals(fd):
    bad = [dict(k=None), dict(v=None), dict(sl=None), dict(acc=None), dict(al=None), dict(out=None), dict(B=-1),
           dict(h=0), dict(page=0), dict(T=0), dict(ma=0), dict(k=A + 8), dict(out=3 * A), dict(out=3 * A + 4),
           dict(out=5 * A), dict(out=4 * A), dict(tl=7 * A, out=7 * A), dict(table=8 * A), dict(acc=A + 2),
           dict(table=8 * A, blocks=2, pages=0), dict(opts=opts(fd, kv_dtype=-1))]
    for over in bad:
        assert compact(fd, **over) == fd.FD_ERR_INVALID_ARG, over
    for over in (dict(d=96), dict(T=257), dict(ma=257), dict(B=5000),
                 dict(table=8 * A, blocks=1 << 20, page=1 << 12, pages=4)):
        assert compact(fd, **over) == fd.FD_ERR_UNSUPPORTED, over
    assert compact(fd, B=0, k=None) == fd.FD_OK


def tree(fd, paged=False, **over):
    a = dict(q=A, k=A, v=A, table=A, blocks=4, mask=A, ms=8, tl=None, sl=A, slh=None, B=2, T=8, hq=8, hkv=2, d=128, smax=64,
             page=16, pages=8, scale=0.1, o=A, lse=A, ws=A, wsb=1 << 40, opts=None)
    a.update(over)
    keys = ["q", "k", "v"] + (["table", "blocks"] if paged else []) + ["mask", "ms", "tl", "sl", "slh", "B", "T", "hq", "hkv", "d"]
    keys += ["page", "pages"] if paged else ["smax"]
    keys += ["scale", "o", "lse", "ws", "wsb", "opts"]
    return (fd._lib.fd_tree_decode_paged if paged else fd._lib.fd_tree_decode)(*[a[k] for k in keys], None)


@pytest.mark.parametrize("paged", [False, True])
def test_tree_refusals(fd, paged):
    long = (ctypes.c_int32 * 2)(10, 65)
    neg = (ctypes.c_int32 * 2)(10, -1)
    bad = [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(ws=None), dict(q=A + 8), dict(k=A + 8), dict(o=A + 4),
           dict(ws=A + 16), dict(mask=A + 4), dict(tl=A + 2), dict(sl=A + 2), dict(lse=A + 2), dict(B=-1), dict(T=0), dict(hq=6, hkv=4),
           dict(hkv=0), dict(ms=7), dict(ms=-8), dict(T=65, ms=65), dict(slh=ctypes.addressof(long)), dict(slh=ctypes.addressof(neg)),
           dict(opts=opts(fd, q_len=2)), dict(opts=opts(fd, q_len=-1)), dict(opts=opts(fd, dtype=3)), dict(opts=opts(fd, kv_dtype=7)),
           dict(opts=opts(fd, num_ctas=2000)), dict(opts=opts(fd, kv_dtype=2, k_scale=float("inf")))]
    bad += [dict(table=None), dict(sl=None), dict(blocks=0), dict(page=0), dict(pages=0)] if paged else [dict(smax=-1)]
    for over in bad:
        assert tree(fd, paged, **over) == fd.FD_ERR_INVALID_ARG, over
    for over in [dict(d=96), dict(T=257, ms=0), dict(T=256, ms=0, hq=34, hkv=2), dict(B=5000)] + (
            [dict(page=24), dict(page=96), dict(page=1 << 16, blocks=1 << 15), dict(page=1 << 16, pages=1 << 15)] if paged
            else [dict(smax=1 << 30)]):
        assert tree(fd, paged, **over) == fd.FD_ERR_UNSUPPORTED, over
    assert tree(fd, paged, wsb=16) == fd.FD_ERR_WORKSPACE_TOO_SMALL
    assert tree(fd, paged, B=0) == fd.FD_OK


def test_tree_workspace_size(fd):
    size = fd.fd_tree_workspace_size
    assert size(1, 1, 8, 8, 128) >= 256
    assert size(4096, 256, 16, 1, 256) >= 256   # 4096 query rows of a kv head
    for args in ((-1, 8, 8, 2, 128), (5000, 8, 8, 2, 128), (1, 0, 8, 2, 128), (1, 257, 8, 2, 128), (1, 8, 6, 4, 128),
                 (1, 8, 8, 0, 128), (1, 8, 8, 2, 96), (1, 256, 34, 2, 128)):
        assert size(*args) == 0, args
    with pytest.raises(fd.FdError):
        fd.make_tree_workspace(1, 300, 8, 8)
