"""Accuracy of the tree attention over long runs of tiles: errors by norm, and scores that grow all along."""
import numpy as np
import pytest
import torch

from spec_util import make_tree_case, pack_mask
from tree_accuracy import NORM_BOUND, attention64, norm_errors

pytestmark = pytest.mark.gpu


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


# (nodes, query heads, kv heads): 16 query rows a kv head, which both softmax groups share; 160, a group's own
ROWS = [(8, 4, 2), (40, 8, 2)]


@pytest.mark.parametrize("T,hq,hkv", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kv,page,ctas", [("bf16", "same", 0, 1), ("f16", "same", 0, 1), ("bf16", "e4m3", 16, 1),
                                                ("bf16", "same", 16, 5), ("f16", "e5m2", 0, 2), ("bf16", "same", 4, 1)])
def test_error_by_norm(fd, T, hq, hkv, D, dtype, kv, page, ctas):
    """Requests short and long, few CTAs: losing the weights' second part, or the flushes of the
    accumulators, would pass the bounds for single elements but not this one.  LSE: the scores'
    2^-16, and sums of some 700 fp32 additions in a thread's turn, 2^-24 each: below 2^-14."""
    lens = [300, 40000, 16500]
    c = make_tree_case(60, 3, T, hq, hkv, D, lens, dtype=dtype, kv=kv, page=page)
    ks, vs = (0.7, 1.3) if kv != "same" else (1.0, 1.0)
    ref, ref_lse = attention64(c, D ** -0.5, ks, vs, device="cuda")
    o, lse = run(fd, c, D ** -0.5, num_ctas=ctas, k_scale=ks, v_scale=vs)
    errors = norm_errors(o, ref)
    print("errors by norm:", ["%.2e" % e for e in errors])
    assert max(errors) <= NORM_BOUND, errors
    assert float((lse.double().cpu() - ref_lse).abs().max()) <= 2.0 ** -14


@pytest.mark.parametrize("T,hq,hkv", [(8, 4, 1), (40, 4, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kv", [("bf16", "same"), ("f16", "same"), ("bf16", "e5m2")])
@pytest.mark.parametrize("L,ctas", [(1100, 1), (9500, 1), (9500, 3)])
def test_scores_that_grow_all_along(fd, T, hq, hkv, D, dtype, kv, L, ctas):
    """Scores that rise from 0 to 107 (2^154 in the weights) over the request, beside rows of a warp
    whose scores fall, stay, or rise by half.  Over 1100 positions every tile moves the running
    maximum and rescales; over 9500 in one CTA the flushed sums' reference falls more than 2^60
    behind and is moved.  V is positive, and for bf16 falls as the weights of the rising rows rise:
    every part of the request counts for as much, and what is lost or scaled wrongly shows.

    Bound, relative since nothing cancels: a score of up to S is off by (D / 16 + 1) steps of 2^-23 S,
    the arguments of the exponentials (of a weight, of the rescaling, of a flush) by 8 roundings of
    2^-24 S / ln 2, a weight by 2^-16; twice, for O and for the sum; accumulators lose 256 2^-23 = 2^-15 at
    most, the fp32 sums as much.  fp16 weights (the MMAs' type, for FP8 caches too) below 2^-33 of the
    largest may be lost, hence V of one size there."""
    S = 107.0
    c = make_tree_case(61, 1, T, hq, hkv, D, [L], dtype=dtype, kv=kv)
    rng = np.random.default_rng(L)
    q = np.array([16.0, -16.0, 0.0, 8.0])[np.arange(T) % 4]
    c["q64"] = np.broadcast_to(q[None, :, None, None], c["q64"].shape).copy()
    c["q"] = torch.from_numpy(c["q64"]).to(c["q"].dtype)
    k = np.linspace(0.0, S / 16.0, L)[:, None, None] + 0.05 * rng.standard_normal((L, 1, D))
    c["k"] = torch.from_numpy(k[None]).float().to(c["k"].dtype)
    c["k64"] = [c["k"][0].float().double().numpy()]
    v = np.abs(rng.standard_normal((L, 1, D)))
    if dtype == "bf16" and kv == "same":
        v = v * np.exp2(70.0 - np.round(16.0 * c["k64"][0].mean((1, 2)) / np.log(2.0)))[:, None, None]
    c["v"] = torch.from_numpy(v[None]).float().to(c["v"].dtype)
    c["v64"] = [c["v"][0].float().double().numpy()]
    S = float(np.abs(c["k64"][0]).mean((1, 2)).max()) * 16.0
    bound = 2 * ((D / 16 + 1) * 2.0 ** -23 * S + 8 * S / np.log(2.0) * 2.0 ** -24 + 2.0 ** -16) + 2.0 ** -14
    ref, ref_lse = attention64(c, 1.0 / D, device="cuda")
    o, lse = run(fd, c, 1.0 / D, num_ctas=ctas)
    off = ((o.double().cpu() - ref).abs() / ref).amax((0, 2, 3))
    assert float(off.max()) <= bound, (bound, off.tolist())
    assert float((lse.double().cpu() - ref_lse).abs().max()) <= bound
