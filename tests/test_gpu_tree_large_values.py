"""Tree attention over large finite V behind weights that fp32 does not hold, and infinities beside them."""
import math

import numpy as np
import pytest
import torch

from spec_util import TYPES, make_tree_case, pack_mask, tree_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


@pytest.mark.parametrize("dtype,kv", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("near", ["first", "last", "spread"])
@pytest.mark.parametrize("L,ctas", [(300, 1), (6000, 0), (6000, 3)])
@pytest.mark.parametrize("bad", [False, True])
def test_large_finite_values_vanish_and_infinities_stay(fd, dtype, kv, near, L, ctas, bad):
    """Far rows score 256 nats below the near ones, weights of 2^-369, and hold numbers near their type's largest (bf16:
    2^112): 0 in fp32, whichever tile or CTA has them.  An infinity among them stays one.
    Bound: the near rows' weights are equal; of each of n additions and of each CTA's logarithm of a sum of weights (up to
    8: 2^-21 of it) 2^-20 is allowed."""
    if bad and kv == "e4m3":
        pytest.skip("the type has no infinity")
    T, D = 5, 128
    c = make_tree_case(3, 1, T, 4, 2, D, [L], dtype=dtype, kv=kv)
    top = np.zeros(L, dtype=bool)
    top[{"first": slice(0, 3), "last": slice(L - T - 3, L - T), "spread": slice(5, L - T, L // 6)}[near]] = True
    kvt = TYPES[dtype if kv == "same" else kv]
    k, v = np.zeros((L, 2, D)), np.random.default_rng(7).standard_normal((L, 2, D))
    k[~top] = -1.0
    v[~top] = 2.0 ** 112 if kvt is torch.bfloat16 else torch.finfo(kvt).max
    v[~top, :, 1::2] *= -1
    v[top, :, 96:] = 0.0
    if bad:
        far = np.nonzero(~top)[0]
        far = far[far < L - T]
        v[far[1], :, 5] = v[far[-2], :, 100] = math.inf
        v[far[-1], :, 6] = -math.inf
        v[far[0], :, 20], v[far[-1], :, 20] = math.inf, -math.inf
    c["q"] = torch.full_like(c["q"], 4.0)
    for name, x in (("k", k), ("v", v)):
        t = torch.from_numpy(x).to(kvt)
        c[name][0] = t
        c[name + "64"] = [t.double().numpy()]
    mask = torch.from_numpy(pack_mask(c["vis"]).view(np.int64)).cuda()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    o, lse = fd.fd_tree_decode(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), lens, mask, scale=0.5, num_ctas=ctas)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    ref, ref_lse, _, _ = tree_attention(c["q"].double().numpy(), c["k64"], c["v64"], c["vis"], [L], c["trees"], 0.5)
    assert np.abs(lse - ref_lse).max() <= 2.0 ** -18
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    inf, fin = np.isinf(ref), np.isfinite(ref)
    assert bool(inf.any()) == bad and np.array_equal(o[inf], ref[inf])
    bound = ((top.sum() + 16) * 2.0 ** -20 * np.abs(c["v64"][0][top]).mean(0)).repeat(2, 0)[None, None] + 2.0 ** -149
    off = np.abs(o[fin] - ref[fin])
    assert (off <= np.broadcast_to(bound, o.shape)[fin]).all(), off.max()
