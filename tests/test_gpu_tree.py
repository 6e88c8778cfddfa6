"""fd_tree_decode and fd_tree_decode_paged on the GPU, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from spec_util import check_tree, make_tree_case, pack_mask, tree_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(fd, c, scale, mask="own", **kw):
    if mask == "own":
        mask = torch.from_numpy(pack_mask(c["vis"]).view(np.int64)).cuda()
    if "trees_dev" not in kw:
        kw["tree_lens"] = i32(c["trees"]) if any(t != c["q"].shape[1] for t in c["trees"]) else None
    args = dict(tree_mask=mask, scale=scale, **kw)
    q, k, v = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    if c["page"]:
        return fd.fd_tree_decode_paged(q, k, v, c["block_table"].cuda(), i32(c["lens"]), **args)
    return fd.fd_tree_decode(q, k, v, i32(c["lens"]), **args)


def want(c, scale, ks=1.0, vs=1.0):
    return tree_attention(c["q64"], c["k64"], c["v64"], c["vis"], c["lens"], c["trees"], scale * ks, vs)


# lengths: empty, one token, fewer tokens than nodes, inside / at / past a tile, several tiles
LENS = [0, 1, 5, 13, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (4, 4, 13), (8, 2, 7), (14, 2, 20), (16, 2, 16), (3, 3, 64), (8, 2, 33),
                                      (16, 2, 30), (16, 1, 40), (5, 1, 130)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_shapes(fd, hq, hkv, T, D):
    """Group sizes and trees from 1 to 650 query rows a kv head, over every kind of length."""
    c = make_tree_case(hq * 100 + T, len(LENS), T, hq, hkv, D, LENS)
    check_tree(*run(fd, c, D ** -0.5), want(c, D ** -0.5))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 192])
@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(fd, page, kv, D):
    c = make_tree_case(page, 6, 17, 8, 2, D, [0, 1, 17, 130, 256, 401], page=page, kv=kv)
    check_tree(*run(fd, c, 0.11, k_scale=0.5, v_scale=2.0), want(c, 0.11, *((0.5, 2.0) if kv != "same" else ())))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv", ["same", "e4m3", "e5m2"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [6, 40])
def test_types(fd, dtype, kv, D, T):
    c = make_tree_case(7, 3, T, 8, 2, D, [50, 200, 129], dtype=dtype, kv=kv)
    ks, vs = (0.7, 1.3) if kv != "same" else (1.0, 1.0)
    check_tree(*run(fd, c, D ** -0.5, k_scale=ks, v_scale=vs), want(c, D ** -0.5, ks, vs))


@pytest.mark.parametrize("T", [1, 20, 70])
@pytest.mark.parametrize("ctas", [0, 1, 3, 4, 7, 40])
@pytest.mark.parametrize("D,kv,page", [(64, "same", 0), (128, "same", 0), (256, "same", 64), (128, "e4m3", 16), (256, "e5m2", 0),
                                       (128, "same", 4)])
def test_long_requests_split_many_ways(fd, T, ctas, D, kv, page):
    """Few CTAs: long runs of tiles, several segments a CTA, every kind of partial; flushed accumulators (5000 positions)."""
    lens = [700, 1, 5000, 0, 300]
    c = make_tree_case(T, 5, T, 4, 1, D, lens, kv=kv, page=page)
    check_tree(*run(fd, c, 0.09, num_ctas=ctas), want(c, 0.09))


@pytest.mark.parametrize("page", [0, 16])
def test_ragged_trees(fd, page):
    T = 40
    c = make_tree_case(5, 6, T, 8, 2, 128, [100, 100, 7, 200, 0, 300], trees=[0, 1, 40, 17, 40, 39], page=page)
    check_tree(*run(fd, c, 0.09), want(c, 0.09))


@pytest.mark.parametrize("kind", ["empty rows", "all", "none", "random", "without self"])
@pytest.mark.parametrize("lens", [[20, 64, 12], [150, 129, 300]])
def test_masks(fd, kind, lens):
    """Masks that are no tree: rows that see nothing (without context: no output), every node, others but not themselves."""
    T = 20
    c = make_tree_case(11, 3, T, 8, 2, 64, lens)
    rng = np.random.default_rng(1)
    vis = c["vis"]
    if kind == "empty rows":
        vis[:, ::3] = False
    elif kind in ("all", "none"):
        vis[:] = kind == "all"
    elif kind == "random":
        vis[:] = rng.random(vis.shape) < 0.3
    else:
        vis &= ~np.eye(T, dtype=bool)
    check_tree(*run(fd, c, 0.1), want(c, 0.1))


def test_one_mask_for_all_and_bits_behind_the_tree(fd):
    T = 70
    c = make_tree_case(12, 3, T, 4, 2, 64, [80, 300, 129], trees=[70, 5, 66])
    c["vis"][:] = c["vis"][0]
    w = want(c, 0.1)
    words = pack_mask(c["vis"])
    one = torch.from_numpy(words[0].view(np.int64)).cuda()
    check_tree(*run(fd, c, 0.1, mask=one), w)
    words[..., 1] |= np.uint64(0xFFFFFFFFFFFFFFFF) << np.uint64(6)   # nodes 70 .. 127 do not exist
    check_tree(*run(fd, c, 0.1, mask=torch.from_numpy(words).cuda()), w)


@pytest.mark.parametrize("T,hq,hkv", [(4, 8, 2), (16, 4, 4), (33, 8, 1)])
def test_no_mask_is_a_causal_chain(fd, T, hq, hkv):
    c = make_tree_case(13, 4, T, hq, hkv, 128, [3, 50, 200, 129])
    c["vis"][:] = np.tril(np.ones((T, T), dtype=bool))
    got = run(fd, c, 0.1, mask=None)
    check_tree(*got, want(c, 0.1))
    if T * hq // hkv <= 16:   # the same call of the decode entry point
        q, k, v = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
        for b in range(4):   # NaN padding is not read by either
            o, l = fd.fd_decode(q, k, v, i32(c["lens"]), scale=0.1)
        w = want(c, 0.1)
        check_tree(o, l, (w[0], w[1], 2 * w[2], 2 * w[3]))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-8, 3.0])
def test_scales(fd, scale):
    c = make_tree_case(14, 2, 9, 4, 2, 64, [40, 200])
    check_tree(*run(fd, c, scale), want(c, scale))


@pytest.mark.parametrize("D,T", [(64, 12), (128, 12), (256, 12), (128, 50)])
@pytest.mark.parametrize("what", ["hidden node", "seen by some", "infinite value"])
def test_not_a_number_in_masked_places(fd, what, D, T):
    """What a row does not see does not reach it, NaN and infinities included; what it sees does."""
    lens = [140, 30, 400]
    c = make_tree_case(15, 3, T, 8, 2, D, lens)
    for b, L in enumerate(lens):
        node = T // 2
        if what == "hidden node":
            c["vis"][b, :, node] = False
        pos = L - T + node
        for name in ("k", "v"):
            bad = float("inf") if what == "infinite value" else float("nan")
            if what == "infinite value" and name == "k":
                continue   # the score would be infinite: its weight is not a number in any form
            c[name][b, pos, 1, 3::7] = bad
            c[name + "64"][b][pos, 1, 3::7] = bad
    check_tree(*run(fd, c, 0.1), want(c, 0.1))


def test_not_a_number_that_every_row_sees(fd):
    c = make_tree_case(16, 2, 6, 4, 2, 128, [300, 200])
    c["v"][0, 17, 0, 5] = c["v64"][0][17, 0, 5] = float("nan")
    c["k"][1, 150, 1, 9] = c["k64"][1][150, 1, 9] = float("nan")
    check_tree(*run(fd, c, 0.1), want(c, 0.1))


def test_large_scores(fd):
    """Scores of several thousands: the weights stay finite and the running maximum moves in every tile."""
    c = make_tree_case(17, 2, 8, 4, 2, 64, [400, 257], std=60.0)
    order = np.argsort(c["k64"][0][:, 0, 0])
    check_tree(*run(fd, c, 1.0), want(c, 1.0))
    assert order.size


def test_outputs_without_lse_and_given_buffers(fd):
    c = make_tree_case(18, 2, 8, 4, 2, 64, [40, 200])
    w = want(c, 0.1)
    out = torch.full((2, 8, 4, 64), float("nan"), device="cuda")
    lse = torch.full((2, 8, 4), float("nan"), device="cuda")
    got = run(fd, c, 0.1, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check_tree(out, lse, w)
    o, l = run(fd, c, 0.1, lse=False)
    assert l is None
    check_tree(o, None, w)


def test_bad_device_values_are_reported(fd):
    c = make_tree_case(19, 2, 8, 4, 2, 64, [40, 60], page=16)
    ws = fd.make_tree_workspace(2, 8, 4, 2, 64)
    w = want(c, 0.1)
    check_tree(*run(fd, c, 0.1, workspace=ws), w)
    assert fd.fd_get_device_error(ws) == fd.FD_OK
    good = c["block_table"].clone()
    c["block_table"][1, 2] = 1000
    o, l = run(fd, c, 0.1, workspace=ws)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_DEVICE_INPUT
    check_tree(o[:1], l[:1], tuple(x[:1] for x in w))   # the other request is untouched
    c["block_table"] = good
    trees = c["trees"]
    c["trees"] = [8, 9]
    o, l = run(fd, c, 0.1, workspace=ws)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_DEVICE_INPUT
    check_tree(o, l, w)   # 9 nodes of 8: clamped
    c["trees"], lens = trees, c["lens"]
    c["lens"] = [40, -1]
    o, l = run(fd, c, 0.1, workspace=ws)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_DEVICE_INPUT
    assert not o[1].any() and torch.isneginf(l[1]).all()
    c["lens"] = lens
    check_tree(*run(fd, c, 0.1, workspace=ws), w)
    assert fd.fd_get_device_error(ws) == fd.FD_OK


def test_python_refusals(fd):
    c = make_tree_case(20, 2, 8, 4, 2, 64, [40, 60])
    q, k, v, lens = c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), i32(c["lens"])
    mask = torch.from_numpy(pack_mask(c["vis"]).view(np.int64)).cuda()
    for bad in (dict(q=q[:, 0]), dict(q=c["q"]), dict(k=k.half()), dict(k=k[:1]), dict(v=v[:, :, :1]), dict(m=mask.int()),
                dict(m=mask[:, :4]), dict(m=mask.cpu()), dict(t=i32([8])), dict(l=lens.long()), dict(l=lens[:1])):
        a = dict(q=q, k=k, v=v, l=lens, m=mask, t=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            fd.fd_tree_decode(a["q"], a["k"], a["v"], a["l"], a["m"], tree_lens=a["t"])
    with pytest.raises(fd.FdError):
        fd.fd_tree_decode(q, k, v, lens, mask, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fd.fd_tree_decode_paged(q, k, v, None, lens, mask)


@pytest.mark.parametrize("page,kv,T,D", [(0, "same", 8, 128), (16, "same", 50, 128), (4, "same", 8, 64), (0, "e4m3", 40, 128),
                                         (64, "same", 8, 256)])
def test_a_starved_wait_times_out_and_the_context_survives(fd, page, kv, T, D):
    """A first tile that never arrives: every role gives up, the tensor memory is freed, the host
    reads FD_ERR_TIMEOUT, and the same workspace serves the next call."""
    c = make_tree_case(21, 2, T, 8, 2, D, [700, 300], page=page, kv=kv)
    ws = fd.make_tree_workspace(2, T, 8, 2, D)
    run(fd, c, 0.1, workspace=ws, num_ctas=4, flags=fd.FD_FLAG_TEST_STARVE_FIRST_TILE, wait_timeout_ns=50_000_000)
    assert fd.fd_get_device_error(ws) == fd.FD_ERR_TIMEOUT
    check_tree(*run(fd, c, 0.1, workspace=ws, num_ctas=4), want(c, 0.1))
    assert fd.fd_get_device_error(ws) == fd.FD_OK


@pytest.mark.parametrize("page,kv", [(16, "same"), (4, "same"), (16, "e4m3"), (2, "e4m3")])
def test_pages_past_32_bit_offsets(fd, page, kv):
    """Pages whose element offsets pass 2^32 (a pool of 2.3 M slots x 8 heads x 256)."""
    from spec_util import TYPES
    hkv, D, slots = 8, 256, 2300 * 1024
    pages = slots // page
    kt = TYPES["bf16" if kv == "same" else kv]
    pool = [torch.zeros(pages, page, hkv, D, dtype=torch.uint8 if kv != "same" else torch.int16, device="cuda").view(kt) for _ in range(2)]
    c = make_tree_case(30, 2, 6, 16, hkv, D, [70, 33], kv=kv)
    need = [-(-n // page) for n in c["lens"]]
    table = torch.zeros(2, max(need), dtype=torch.int32)
    at = pages - sum(need)                  # the pool's last pages
    for b in range(2):
        for j in range(need[b]):
            table[b, j] = at
            n = min(page, c["lens"][b] - j * page)
            for t, x in zip(pool, (c["k"], c["v"])):
                view = torch.uint8 if kv != "same" else torch.int16
                t.view(view)[at, :n] = x.view(view)[b, j * page:j * page + n].cuda()
            at += 1
    mask = torch.from_numpy(pack_mask(c["vis"]).view(np.int64)).cuda()
    got = fd.fd_tree_decode_paged(c["q"].cuda(), *pool, table.cuda(), i32(c["lens"]), mask, scale=0.06)
    check_tree(*got, want(c, 0.06))


def test_largest_trees_and_groups(fd):
    """256 nodes; 4096 query rows of one kv head."""
    c = make_tree_case(31, 1, 256, 2, 1, 64, [300])
    check_tree(*run(fd, c, 0.1), want(c, 0.1))
    c = make_tree_case(32, 1, 64, 64, 1, 64, [200], dtype="f16")
    check_tree(*run(fd, c, 0.1), want(c, 0.1))


def test_fp8_rows_of_every_magnitude(fd):
    """FP8 caches take a bf16 query as fp16 rows over a power of two: rows from 2^-100 to 2^100, zero rows, mixed rows."""
    c = make_tree_case(33, 2, 8, 4, 2, 128, [200, 70], kv="e4m3")
    powers = torch.tensor([-100, -30, 0, 20, 60, 100, -126, 8], dtype=torch.float32)
    q = c["q"].float() * torch.exp2(powers)[None, :, None, None]
    q[:, 3, 1] = 0
    q[:, 7, :, ::2] *= 2.0 ** -20
    for scale_power in (0, -100, 100):       # the scale brings some of them near 1
        c["q"] = (q / 4).to(torch.bfloat16)
        c["q64"] = c["q"].double().numpy()
        scale = 2.0 ** scale_power
        w = want(c, scale)
        rows = [i for i in range(8) if np.isfinite(w[2][:, i]).all() and np.abs(w[1][:, i]).max() < 1e4]
        got = run(fd, c, scale)
        assert rows
        check_tree(got[0][:, rows], got[1][:, rows], tuple(x[:, rows] for x in w))


@pytest.mark.parametrize("kv,page,T", [("e4m3", 0, 12), ("e4m3", 16, 50), ("e5m2", 4, 12)])
def test_fp8_codes_that_are_no_numbers_in_masked_places(fd, kv, page, T):
    c = make_tree_case(34, 2, T, 8, 2, 128, [140, 400], kv=kv, page=page)
    for b, L in enumerate(c["lens"]):
        pos = L - T + T // 2                  # seen by its descendants and itself
        at = (int(c["block_table"][b, pos // page]), pos % page) if page else (b, pos)
        for name in ("k", "v"):
            c[name].view(torch.uint8)[at[0], at[1], 1, 3::7] = 0x7F   # NaN in both types
            c[name + "64"][b][pos, 1, 3::7] = float("nan")
        if kv == "e5m2":                      # and an infinity that few see
            c["v"].view(torch.uint8)[at[0], at[1], 0, 5] = 0x7C
            c["v64"][b][pos, 0, 5] = float("inf")
    check_tree(*run(fd, c, 0.1), want(c, 0.1))
