"""Tree attention on values that its other tests do not hold: infinities among
the context's V, and a length next to 2^31."""
import numpy as np
import pytest
import torch

from spec_util import check_tree, make_tree_case, pack_mask, tree_attention

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(fd, c, scale, **kw):
    mask = torch.from_numpy(pack_mask(c["vis"]).view(np.int64)).cuda()
    q, k, v = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    if c["page"]:
        return fd.fd_tree_decode_paged(q, k, v, c["block_table"].cuda(), i32(c["lens"]), mask, scale=scale, **kw)
    return fd.fd_tree_decode(q, k, v, i32(c["lens"]), mask, scale=scale, **kw)


def put(c, name, b, pos, head, dim, value):
    """Set one element of a case's cache, in the tensor and in its 64-bit form."""
    page = c["page"]
    at = (int(c["block_table"][b, pos // page]), pos % page) if page else (b, pos)
    t = c[name]
    if t.element_size() == 1:
        t.view(torch.uint8)[at[0], at[1], head, dim] = int(torch.tensor(value).to(t.dtype).view(torch.uint8))
    else:
        t[at[0], at[1], head, dim] = value
    c[name + "64"][b][pos, head, dim] = value


# The bounds of tree_attention hold for the finite elements; the others have to be equal.  In a dim with
# an infinity that a row sees, its output is that infinity (weights are above 0 however small), and NaN
# with both signs or with a NaN.
@pytest.mark.parametrize("std", [1.5, 25.0])   # 25: scores hundreds apart, weights far below fp32's least
@pytest.mark.parametrize("ctas", [0, 1, 3])
@pytest.mark.parametrize("D,T,dtype,kv,page", [(128, 12, "bf16", "same", 0), (128, 50, "bf16", "same", 16), (64, 12, "f16", "same", 0),
                                               (256, 12, "bf16", "same", 0), (128, 12, "f16", "e5m2", 16), (64, 50, "bf16", "e5m2", 0),
                                               (256, 40, "f16", "e5m2", 4), (128, 12, "f16", "same", 4)])
def test_infinities_in_the_context(fd, D, T, dtype, kv, page, ctas, std):
    lens = [140, 70, 4500, T + 1]
    c = make_tree_case(40, 4, T, 8, 2, D, lens, dtype=dtype, kv=kv, page=page, std=std)
    for b, L in enumerate(lens):
        base = L - T
        for head in range(2):
            last = base - 1
            put(c, "v", b, 0, head, 1, INF)
            put(c, "v", b, last, head, 2, -INF)
            put(c, "v", b, last // 3, head, 3, INF)          # both signs, in tiles of their own in the long request
            put(c, "v", b, last, head, 3, -INF if last else INF)
            put(c, "v", b, last // 2, head, 4, NAN)
            put(c, "v", b, last // 2, head, D - 1, -INF)
            node = base + T // 2                              # one sign in the context, the other in a node that few rows see
            put(c, "v", b, last // 4, head, 5, INF)
            put(c, "v", b, node, head, 5, -INF)
            put(c, "v", b, node, head, 6, INF)
            for pos in range(0, base, 3):
                put(c, "v", b, pos, head, D // 2, INF)
    check_tree(*run(fd, c, 0.1, num_ctas=ctas), tree_attention(c["q64"], c["k64"], c["v64"], c["vis"], lens, c["trees"], 0.1))


def test_a_length_next_to_2_31(fd):
    """2^31 - 64 positions behind a table that names 8 pages again and again: the positions of a page
    weigh as often as it is named.  A thread adds up to 2^31 / 128 / 152 = 110000 tiles' sums in fp32, 2^-24
    each, in the sum of the weights and in O: 2 x 110000 x 2^-24 = 1.3e-2 at most, with the rest 1.4e-2; V is
    positive, so the bound is relative."""
    D, T, page, pages, blocks = 64, 2, 64, 9, (1 << 25) - 1
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(1, T, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn(pages, page, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(pages, page, 1, D, generator=g, device="cuda").abs().to(torch.bfloat16)
    table = torch.randint(0, 8, (1, blocks), generator=g, device="cuda", dtype=torch.int32)
    table[0, -1] = 8                                          # the nodes' page: its last two positions
    lens = i32([blocks * page])
    ws = fd.make_tree_workspace(1, T, 1, 1, D)
    o, lse = fd.fd_tree_decode_paged(q, k, v, table, lens, workspace=ws, scale=0.125)
    assert fd.fd_get_device_error(ws) == fd.FD_OK
    often = torch.bincount(table[0], minlength=pages).double().repeat_interleave(page).repeat(T, 1)
    often[0, -1] = 0                                          # node 0 does not see node 1
    s = (q[0, :, 0].double() @ k.view(-1, D).double().T) * 0.125 + often.log()
    ref = torch.softmax(s, -1) @ v.view(-1, D).double()
    assert float(((o[0, :, 0].double() - ref).abs() / ref).max()) <= 1.4e-2
    assert float((lse[0, :, 0].double() - torch.logsumexp(s, -1)).abs().max()) <= 1.4e-2
