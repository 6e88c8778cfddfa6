"""fd_window_decode, fd_decode4 and their paged forms on the GPU, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import longcontext_util as u
from spec_util import check_tree as check

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "e4m3", "e5m2", "e2m1"]


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def scales(kv):
    return (0.7, 1.3) if kv in ("e4m3", "e5m2", "e2m1") else (1.0, 1.0)


def both(fd, c, scale, **kw):
    ks, vs = scales(c["kv"])
    check(*u.run(fd, c, scale, k_scale=ks, v_scale=vs, **kw), u.want(c, scale, ks, vs))


# lengths: empty, one token, fewer tokens than new ones, inside / at / past a tile, several tiles
LENS = [0, 1, 2, 5, 15, 16, 17, 31, 32, 33, 64, 65, 200]


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (4, 4, 3), (8, 2, 1), (14, 2, 1), (6, 2, 5), (16, 1, 1), (3, 3, 16), (12, 4, 4), (10, 5, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", KINDS)
def test_shapes(fd, hq, hkv, T, D, kv):
    """Groups and new tokens from 1 to 16 columns, over every kind of length; whole caches in 4 bits, else a window of 40 and 3 sinks."""
    more = {} if kv == "e2m1" else dict(window=40, sinks=3)
    both(fd, u.make_case(hq * 100 + T, len(LENS), T, hq, hkv, D, LENS, kv=kv, **more), D ** -0.5)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 33, 64, 100, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 17, 32, 150, 5000])
@pytest.mark.parametrize("kv,T", [("e2m1", 1), ("e2m1", 5), ("bf16", 1), ("f16", 6), ("e4m3", 1), ("bf16", 3)])
def test_windows(fd, window, sinks, kv, T):
    """Windows and sinks that end anywhere in a tile, overlap, and pass the lengths."""
    both(fd, u.make_case(window * 7 + sinks, 8, T, 8, 4, 128, [0, 1, 4, 40, 110, 150, 181, 300], kv=kv, window=window, sinks=sinks), 0.09)


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 24, 64, 100])
@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("D,T", [(64, 1), (128, 3), (256, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5)])
def test_pages(fd, page, kv, D, T, window, sinks):
    """Any page size; the pages that nobody sees have no entry."""
    both(fd, u.make_case(page, 5, T, 6, 2, D, [0, 1, 17, 130, 301], kv=kv, page=page, window=window, sinks=sinks), 0.11)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 3])
def test_query_types(fd, dtype, kv, D, T):
    """bf16 and fp16 queries over narrower caches; rows of very different sizes."""
    c = u.make_case(7, 3, T, 8, 2, D, [50, 200, 129], kv=kv, dtype=dtype)
    f = torch.exp2(torch.tensor([0.0, -3.0, 2.0, -8.0, 1.0, -12.0, 0.0, -1.0]))[None, None, :, None]
    c["q"] = (c["q"].float() * f).to(c["q"].dtype)
    c["q64"] = c["q"].double().numpy()
    both(fd, c, D ** -0.5)


@pytest.mark.parametrize("dtype,kv", [("bf16", "e2m1"), ("bf16", "bf16"), ("f16", "e2m1"), ("bf16", "e5m2")])
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -60, 2.0 ** 60, 2.0 ** -120, 2.0 ** 119])
def test_query_sizes(fd, dtype, kv, factor):
    """Queries near either end of bf16 (fp16: 2^-14 and 2^13), with the scale that brings the scores back."""
    if dtype == "f16":
        factor = {0.0: 0.0, 2.0 ** -60: 2.0 ** -8, 2.0 ** 60: 2.0 ** 8, 2.0 ** -120: 2.0 ** -12, 2.0 ** 119: 2.0 ** 12}[factor]
    c = u.make_case(8, 2, 1, 8, 2, 128, [70, 33], kv=kv, dtype=dtype)
    c["q"] = (c["q"].float() * factor).to(c["q"].dtype)
    c["q64"] = c["q"].double().numpy()
    ks, vs = scales(kv)
    scale = float(np.float32(0.09 / factor)) if factor else 0.09
    check(*u.run(fd, c, scale, k_scale=ks, v_scale=vs), u.want(c, scale, ks, vs))


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-6, 2.0])
@pytest.mark.parametrize("kv,T", [("e2m1", 1), ("bf16", 4), ("e4m3", 1)])
def test_scales(fd, scale, kv, T):
    both(fd, u.make_case(9, 3, T, 8, 2, 128, [70, 33, 5], kv=kv, window=30, sinks=2), scale)


@pytest.mark.parametrize("ctas", [0, 1, 2, 3, 7, 40])
@pytest.mark.parametrize("hq,hkv,T", [(4, 1, 1), (8, 4, 1), (4, 2, 4), (16, 4, 4)])
@pytest.mark.parametrize("D,kv,page", [(64, "bf16", 0), (128, "f16", 0), (256, "bf16", 64), (128, "e4m3", 16), (64, "e5m2", 0),
                                       (128, "e2m1", 16), (256, "e2m1", 0), (64, "e2m1", 64)])
def test_split_many_ways(fd, ctas, hq, hkv, T, D, kv, page):
    """Few CTAs: long runs of tiles, several segments a warp, every kind of partial."""
    both(fd, u.make_case(T, 6, T, hq, hkv, D, [700, 1, 3000, 0, 300, 40], kv=kv, page=page, window=1500, sinks=4), 0.09, num_ctas=ctas)


@pytest.mark.parametrize("B", [200, 700])
@pytest.mark.parametrize("kv", ["e2m1", "e4m3"])
def test_many_requests(fd, B, kv):
    """More requests than a CTA has threads in one scan, most of them empty or short."""
    rng = np.random.default_rng(B)
    lens = (rng.integers(0, 2, B) * rng.integers(0, 60, B)).tolist()
    both(fd, u.make_case(B, B, 1, 2, 1, 64, lens, kv=kv, page=16), 0.125)


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (16, 1, 1), (2, 2, 8), (5, 1, 2)])
@pytest.mark.parametrize("D,kv", [(64, "f16"), (128, "e2m1"), (256, "e2m1"), (128, "bf16"), (256, "e5m2")])
def test_many_partials(fd, hq, hkv, T, D, kv):
    """Few segments that many CTAs share: more partials than are added at once, by one thread or by several."""
    both(fd, u.make_case(D + T, 2, T, hq, hkv, D, [9000, 2500], kv=kv, window=8000, sinks=3), D ** -0.5)


@pytest.mark.parametrize("B,hq,hkv,T", [(40, 8, 8, 1), (75, 8, 4, 1), (150, 6, 6, 2), (40, 32, 16, 2), (152, 4, 1, 4)])
@pytest.mark.parametrize("D,kv,page", [(64, "bf16", 16), (128, "e4m3", 0), (128, "e2m1", 16), (256, "e2m1", 0), (64, "e5m2", 0)])
def test_short_segments(fd, B, hq, hkv, T, D, kv, page):
    """Segments of few tiles, from one to many a CTA, empty requests among them."""
    rng = np.random.default_rng(B + D)
    lens = (rng.integers(0, 4, B).clip(0, 1) * rng.integers(1, 150, B)).tolist()
    both(fd, u.make_case(B, B, T, hq, hkv, D, lens, kv=kv, page=page, window=100, sinks=2), D ** -0.5)


def test_largest_batch(fd):
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 4, 4096).tolist()
    both(fd, u.make_case(4, 4096, 1, 1, 1, 64, lens, kv="e2m1"), 0.125)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("T,hq", [(3, 2), (3, 8), (7, 4)])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_what_a_token_does_not_see_does_not_reach_it(fd, kv, T, hq, bad):
    """NaN or infinity in K and V at the last position and at the window's first, which only some new tokens see: rows
    that do not see them are as without, the others NaN (K, or V with NaN)."""
    if kv == "e2m1" and bad == "inf":
        pytest.skip("the type has no infinity")
    if kv == "e4m3" and bad == "inf":
        pytest.skip("the type has no infinity")
    L, W, S = 120, 40, 5
    c = u.make_case(21, 1, T, hq, 2, 128, [L], kv=kv, window=W, sinks=S)
    places = [L - 1, L - T - W + 1]    # seen by the last token, by the first
    clean = u.want(c, 0.09, *scales(kv))
    x = math.nan if bad == "nan" else math.inf
    for t in places:
        for i, name in enumerate(("k64", "v64")):
            if bad == "inf" and not i:
                continue
            c[name][0][t] = x
            pool = c["pool"]
            if kv == "e2m1":
                pool[2 * i + 1][0, :, t] = 0x7F
            else:
                pool[i][0, t] = torch.tensor(x).to(pool[i].dtype)
    ks, vs = scales(kv)
    o, lse = u.run(fd, c, 0.09, k_scale=ks, v_scale=vs)
    ref = u.want(c, 0.09, ks, vs)
    check(o, lse, ref)
    fine = [i for i in range(T) if not any(u.sees(L, T, i, W, S)[t] for t in places)]
    if T > 2:
        assert fine
    assert np.array_equal(ref[0][0, fine], clean[0][0, fine])


@pytest.mark.parametrize("kv", ["bf16", "f16", "e5m2"])
@pytest.mark.parametrize("hq,T", [(2, 1), (16, 1), (4, 3)])
def test_visible_infinities(fd, kv, hq, T):
    """An infinite V element makes its dim infinite however small its weight, of both signs NaN; split over CTAs too."""
    L = 900
    c = u.make_case(22, 1, T, hq, 2, 64, [L], kv=kv, window=2000, std=6.0)
    for t, d, x in ((3, 5, math.inf), (700, 5, math.inf), (10, 9, -math.inf), (20, 11, math.inf), (850, 11, -math.inf), (400, 20, math.nan)):
        c["v64"][0][t, :, d] = x
        c["pool"][1][0, t, :, d] = torch.tensor(x).to(c["pool"][1].dtype)
    for ctas in (0, 1):
        o, _ = u.run(fd, c, 1.0, num_ctas=ctas, k_scale=1.0, v_scale=1.0)
        assert bool((o[..., 5] == math.inf).all()) and bool((o[..., 9] == -math.inf).all())
        assert bool(o[..., 11].isnan().all()) and bool(o[..., 20].isnan().all())
        assert bool(o[..., [0, 1, 4, 6, 8, 10, 12, 21, 63]].isfinite().all())


@pytest.mark.parametrize("kv", ["bf16", "f16", "e5m2"])
@pytest.mark.parametrize("hq,T", [(1, 1), (8, 2)])
@pytest.mark.parametrize("L,ctas", [(150, 0), (7000, 0), (7000, 3)])
def test_infinities_reach_the_tokens_that_see_them(fd, kv, hq, T, L, ctas):
    """Infinities and NaN anywhere in V of several segments, in ones that a warp has whole, that warps share and that CTAs
    share: every element by the definition, where a weight that 64 bits hold above 0 times an infinity is one."""
    rng = np.random.default_rng(L + T)
    c = u.make_case(31, 3, T, hq, 1, 64, [L, 0, L // 2], kv=kv, window=L // 2, sinks=2)
    for b, n in ((0, L), (2, L // 2)):
        for d in range(0, 64, 5):
            at = int(rng.integers(n - 40 if d % 2 else 0, n))
            x = (math.inf, -math.inf, math.nan)[d % 3]
            c["v64"][b][at, 0, d] = x
            c["pool"][1][b, at, 0, d] = torch.tensor(x).to(c["pool"][1].dtype)
    both(fd, c, 0.125, num_ctas=ctas)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e5m2"])
@pytest.mark.parametrize("T", [1, 3])
def test_large_values_without_weight(fd, kv, T):
    """V of the type's largest numbers at positions whose weights are below 2^-60: they leave no trace beside weights of 1."""
    L = 3000
    c = u.make_case(23, 1, T, 4, 2, 128, [L], kv=kv)
    big = float(torch.finfo(u.TYPES[kv]).max) if kv != "bf16" else 2.0 ** 20
    q = torch.ones_like(c["q"]) * 4
    c["q"], c["q64"] = q, q.double().numpy()
    for name, i, far, near in (("k64", 0, -1.0, 0.0), ("v64", 1, big, 1.0)):
        x = np.full((L, 2, 128), far)
        x[100::977] = near
        c[name][0] = x
        c["pool"][i][0] = torch.from_numpy(x).to(c["pool"][i].dtype)
    o, lse = u.run(fd, c, 0.125)          # scores of -64 nats, 2^-92, and 0: at most 3 rows of weight 1 a token
    assert float((o - 1.0).abs().max()) <= 2.0 ** -20
    check(o, lse, u.want(c, 0.125))


@pytest.mark.parametrize("kv", ["bf16", "e2m1"])
@pytest.mark.parametrize("T", [1, 3])
def test_lengths_next_to_2_31(fd, kv, T):
    """A window at the end of a request of 2^31 - 2 tokens: pages of 49981, of which two are seen."""
    page, blocks, W, S = 49981, 42966, 130, 3
    L = page * blocks
    assert L == 2 ** 31 - 2
    c = u.make_case(24, 1, T, 4, 2, 64, [W + T - 1 + S], kv=kv)      # what is seen, one after another
    n = W + T - 1 + S
    pool = [torch.empty(3, *((2, page) if kv == "e2m1" else (page, 2)), t.shape[-1], dtype=t.dtype, device="cuda") for t in c["pool"]]
    for t, x in zip(pool, c["pool"]):
        x = x[0].cuda()
        for row in range(n):
            pos = row if row < S else L - n + row
            pg, slot = (1 if pos < page else 2), pos % page
            if kv == "e2m1":
                t.view(torch.uint8)[pg, :, slot] = x.view(torch.uint8)[:, row]
            else:
                t[pg, slot] = x[row]
    table = torch.full((1, blocks), -5, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = 1, 2
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = c["q"].cuda()
    ks, vs = scales(kv)
    kw = dict(window=W, sinks=S, scale=0.1, k_scale=ks, v_scale=vs)
    ws = fd.make_window_workspace(1, 4, 2, 64, q_len=T)
    o, lse = (fd.fd_decode4_paged(q, fd.Cache4(*pool), table, lens, workspace=ws, **kw) if kv == "e2m1"
              else fd.fd_window_decode_paged(q, *pool, table, lens, workspace=ws, **kw))
    check(o, lse, u.attention(c["q64"], c["k64"], c["v64"], [n], W, S, 0.1 * ks, vs))
    assert fd.fd_get_device_error(ws) == fd.FD_OK


@pytest.mark.parametrize("kv", KINDS)
def test_as_fd_decode(fd, kv):
    """A window over everything is fd_decode, whose cache is in 16 bits or FP8; a 4-bit one is compared with its values in fp16."""
    B, hq, hkv, D, L = 4, 8, 2, 128, 700
    c = u.make_case(31, B, 2, hq, hkv, D, [700, 3, 260, 64], kv=kv, s_max=L)
    q, lens = c["q"].cuda(), torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    if kv == "e2m1":
        k, v = (torch.from_numpy(np.stack([np.concatenate([x, np.zeros((L - len(x), hkv, D))]) for x in c[n]])).half().cuda() for n in ("k64", "v64"))
        o, lse = fd.fd_decode4(q.half(), fd.Cache4(*(t.cuda() for t in c["pool"])), lens, scale=0.09)
        ro, rl = fd.fd_decode(q.half(), k, v, lens, scale=0.09)
    else:
        k, v = (t.cuda() for t in c["pool"])
        o, lse = fd.fd_window_decode(q, k, v, lens, L, 0, scale=0.09)
        ro, rl = fd.fd_decode(q, k, v, lens, scale=0.09)
    # fd_decode's weights keep 16 bits (bf16); both sides' sums and scores are fp32: 2^-14 of values of a few units
    assert float((o - ro).abs().max()) <= 2.0 ** -12 and torch.equal(lse.isinf(), rl.isinf())
    assert float(torch.nan_to_num(lse - rl, 0.0).abs().max()) <= 2.0 ** -12


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq", [2, 16])
def test_error_by_norm(fd, kv, D, hq):
    """Long runs of tiles (one CTA) by norm: roundings of weights (2^-21 and less), of scores of a few units (D 2^-24
    each, 2^-19 of a weight at most) and of tile sums in fp32 (random signs) come to less than 2^-18 of the output's
    norm; a weight in one 16-bit part is 2^-11 or 2^-8 off."""
    L = 20000
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(1, hq, D, device="cuda", generator=g).to(u.TYPES["f16" if kv == "f16" else "bf16"])
    if kv == "e2m1":
        cache = fd.Cache4(*(torch.randint(0, hi, (1, 2, L, w), device="cuda", generator=g, dtype=torch.uint8) for w, hi in
                            ((D // 2, 256), (D // 16, 56), (D // 2, 256), (D // 16, 56))))
        k, v = (torch.from_numpy(u.values4(a.cpu().numpy(), b.cpu().numpy())).cuda()[0] for a, b in (cache[:2], cache[2:]))
        o, lse = fd.fd_decode4(q, cache, None, scale=D ** -0.5, num_ctas=1)
    else:
        k, v = (torch.randn(1, L, 2, D, device="cuda", generator=g).to(u.TYPES[kv]) for _ in range(2))
        o, lse = fd.fd_window_decode(q, k, v, None, L, scale=D ** -0.5, num_ctas=1)
        k, v = k[0].double().transpose(0, 1), v[0].double().transpose(0, 1)
    s = torch.einsum("hgd,hnd->hgn", q.double().view(2, hq // 2, D), k) * D ** -0.5
    ref, top = torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)
    err = float((o.double().view_as(ref) - ref).norm() / ref.norm())
    print(f"{kv} D={D} columns={hq // 2}: {err:.2e}")
    assert err <= 2.0 ** -18
    assert float((lse.double().view_as(top) - top).abs().max()) <= 2.0 ** -17


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
def test_cache_beyond_4_gb(fd, kv):
    """Pages whose rows lie past 2^32 bytes."""
    H, D, page = 8, 128, 64
    row = {"bf16": 2 * D, "e4m3": D, "e2m1": D // 2}[kv]
    pages = 2 ** 32 // (H * page * row) + 40
    if kv == "e2m1":
        pool = [torch.empty(pages, H, page, w, dtype=torch.uint8, device="cuda") for w in (D // 2, D // 16) * 2]
    else:
        pool = [torch.empty(pages, page, H, D, dtype=u.TYPES[kv], device="cuda") for _ in range(2)]
    c = u.make_case(5, 2, 1, 16, H, D, [400, 130], kv=kv, page=page, window=300, sinks=4)
    ids = torch.randperm(35)[: c["pool"][0].shape[0]] + pages - 36
    for t, x in zip(pool, c["pool"]):
        t.view(torch.uint8)[ids.cuda()] = x.view(torch.uint8).cuda()
    table = torch.where(c["table"] >= 0, ids.int()[c["table"].clamp(min=0).long()], c["table"])
    c.update(pool=[types_like(t) for t in pool], table=table)
    ks, vs = scales(kv)
    check(*u.run(fd, c, 0.09, k_scale=ks, v_scale=vs), u.want(c, 0.09, ks, vs))


def types_like(t):
    return t   # already on the GPU: .cuda() keeps it


@pytest.mark.parametrize("kv", ["bf16", "e2m1"])
def test_bad_device_inputs_are_reported(fd, kv):
    c = u.make_case(41, 3, 1, 4, 2, 64, [100, 30, 60], kv=kv, page=16, window=50, sinks=2)
    ws = fd.make_window_workspace(3, 4, 2, 64)
    good = u.want(c, 0.1, *scales(kv))
    ks, vs = scales(kv)
    o, lse = u.run(fd, c, 0.1, workspace=ws, k_scale=ks, v_scale=vs)
    check(o, lse, good)
    assert fd.fd_get_device_error(ws) == fd.FD_OK
    bad = dict(c, table=c["table"].clone(), lens=[100, 30, 60])
    bad["table"][1, 0] = 1 << 20                      # a page outside the pool: page 0 instead
    o, lse = u.run(fd, bad, 0.1, workspace=ws, k_scale=ks, v_scale=vs)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_DEVICE_INPUT
    for b in (0, 2):
        check(o[b:b + 1], lse[b:b + 1], [x[b:b + 1] for x in good])
    assert fd.fd_get_device_error(ws) == fd.FD_OK
    bad = dict(c, lens=[-4, 30, 1 << 30])             # lengths out of range: clamped
    bad["table"] = c["table"].clamp(min=0)
    o, lse = u.run(fd, bad, 0.1, workspace=ws, k_scale=ks, v_scale=vs)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_DEVICE_INPUT
    check(o[1:2], lse[1:2], [x[1:2] for x in good])
    assert not bool(o[0].any()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("kv", ["bf16", "e2m1"])
def test_repeatable_in_graphs_and_on_other_streams(fd, kv):
    """Bitwise the same results from call to call, on another stream, and from two graphs that share a workspace and are
    replayed with other lengths."""
    c = u.make_case(51, 3, 2, 8, 2, 128, [500, 77, 300], kv=kv, page=16, window=200, sinks=4)
    q, pool, table = c["q"].cuda(), [t.cuda() for t in c["pool"]], c["table"].cuda()
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    ws = fd.make_window_workspace(3, 8, 2, 128, q_len=2)
    out, lse = torch.empty(3, 2, 8, 128, device="cuda"), torch.empty(3, 2, 8, device="cuda")

    def call(**kw):
        kw = dict(workspace=ws, scale=0.09, **kw)
        if kv == "e2m1":
            return fd.fd_decode4_paged(q, fd.Cache4(*pool), table, lens, 200, 4, **kw)
        return fd.fd_window_decode_paged(q, *pool, table, lens, 200, 4, **kw)

    a, la = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, lb = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b) and torch.equal(la, lb)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=out, lse=lse)
        graphs.append(g)
    for g in graphs + graphs:
        out.fill_(math.nan)
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)
    lens.copy_(torch.tensor([40, 0, 299]))
    table.clamp_(min=0)
    a, la = call()
    graphs[0].replay()
    assert torch.equal(a.nan_to_num(7.0), out.nan_to_num(7.0)) and torch.equal(la.nan_to_num(7.0), lse.nan_to_num(7.0))


@pytest.mark.parametrize("kv", ["f16", "e2m1"])
def test_outputs_given_lse_left_out_and_workspace_of_a_larger_shape(fd, kv):
    c = u.make_case(61, 2, 1, 8, 2, 64, [90, 33], kv=kv, window=40)
    ws = fd.make_window_workspace(9, 16, 1, 256)
    o, lse = u.run(fd, c, 0.1, workspace=ws)
    out = torch.full_like(o, math.nan)
    o2, none = u.run(fd, c, 0.1, out=out, lse=False, workspace=ws)
    assert none is None and o2 is out and torch.equal(o, out)
    q3 = dict(c, q=c["q"][:, 0])
    o3, l3 = u.run(fd, q3, 0.1, workspace=ws)
    assert o3.shape == (2, 8, 64) and torch.equal(o3, o[:, 0]) and torch.equal(l3, lse[:, 0])
    lens = torch.tensor(c["lens"], dtype=torch.int32)
    u.run(fd, c, 0.1, workspace=ws, seq_lens_host=lens)
    with pytest.raises(fd.FdError):
        u.run(fd, c, 0.1, workspace=ws, seq_lens_host=lens + 1000)
    with pytest.raises(fd.FdError):
        u.run(fd, c, 0.1, workspace=ws[:256])
    with pytest.raises(ValueError):
        u.run(fd, c, 0.1, out=out[:1])
    assert u.run(fd, dict(c, q=c["q"][:0], pool=[t[:0] for t in c["pool"]], lens=[]), 0.1, workspace=ws)[0].shape == (0, 1, 8, 64)


@pytest.mark.parametrize("kv", ["bf16", "e2m1"])
def test_loop(fd, kv):
    """A serving loop: pages from fd_build_tables, new rows into their slots, attention through a window, and the pages
    behind the window given back: against a cache kept in plain lists."""
    rng = np.random.default_rng(3)
    B, hq, hkv, D, page, pages, W, S = 3, 8, 2, 128, 16, 64, 60, 4
    ks, vs = (0.25, 0.5) if kv == "e2m1" else (1.0, 1.0)
    cache = fd.make_cache4(pages, hkv, page, D) if kv == "e2m1" else tuple(torch.full((pages, page, hkv, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    free = rng.permutation(pages).tolist()
    lens, held = i32([0] * B), i32([0] * B)
    ref = [[np.zeros((0, hkv, D))] * 2 for _ in range(B)]
    ws = fd.make_window_workspace(B, hq, hkv, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    returned = 0
    for new in [[130, 5, 70]] + [[1, 1, 1]] * 3 + [[40, 0, 33]] + [[1, 1, 1]] * 20:
        stack = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        stack[:len(free)] = i32(free)
        t = fd.fd_build_tables(lens, i32(new), table, stack, i32([len(free)]), page, pages, sum(new) + 2, held_pages=held, device_status=status)
        free = free[:int(t.free_count)]
        lens, held = t.seq_lens, t.held_pages
        k, v = (torch.randn(sum(new) + 2, hkv, D, device="cuda").bfloat16() for _ in range(2))
        if kv == "e2m1":
            fd.fd_cache_write4(k, v, t.slot_map, cache, k_scale=ks, v_scale=vs, device_status=status)
            values = [u.values4(*u.quantise4(x.cpu(), s)) for x, s in ((k, ks), (v, vs))]
            back = fd.fd_cache_read4(t.slot_map, cache, k_scale=ks, v_scale=vs, device_status=status)
            for x, y, s in zip(back, values, (ks, vs)):
                assert torch.equal(x[:sum(new)].cpu(), torch.from_numpy(y[:sum(new)] * s).bfloat16()) and not bool(x[sum(new):].any())
        else:
            fd.fd_cache_write(k, v, t.slot_map, *cache, device_status=status)
            values = [x.double().cpu().numpy() for x in (k, v)]
        at = 0
        for b in range(B):
            for i in range(2):
                ref[b][i] = np.concatenate([ref[b][i], values[i][at:at + new[b]]])
            at += new[b]
        q = torch.randn(B, 1, hq, D, device="cuda").bfloat16()
        args = dict(window=W, sinks=S, scale=0.1, workspace=ws)
        o, lse = (fd.fd_decode4_paged(q, cache, table, lens, k_scale=ks, v_scale=vs, **args) if kv == "e2m1"
                  else fd.fd_window_decode_paged(q, *cache, table, lens, **args))
        n = [len(r[0]) for r in ref]
        assert lens.tolist() == n
        # values4 and quantise4 leave the tensor's scale to the call
        check(o, lse, u.attention(q.double().cpu().numpy(), [r[0] for r in ref], [r[1] for r in ref], n, W, S, 0.1 * ks, vs))
        # pages that the next token cannot see go back
        entries = table.cpu()
        for b in range(B):
            for j in range(-(-S // page), (n[b] + 1 - W) // page):
                if entries[b, j] >= 0:
                    free.append(int(entries[b, j]))
                    entries[b, j] = -1
                    returned += 1
        table.copy_(entries)
    assert int(status) == 0 and fd.fd_get_device_error(ws) == fd.FD_OK and returned > 5
