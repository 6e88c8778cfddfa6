"""The plain 64-bit forms that the GPU tests compare with, against other forms and hand-made cases (CPU)."""
import numpy as np
import pytest
import torch

import fd_synth as syn
import oracle
from spec_util import fp8_round, make_tree_case, pack_mask, random_tree, tables, tree_attention, tree_visibility


def test_tree_attention_is_the_masked_softmax():
    c = make_tree_case(3, 2, 7, 4, 2, 64, [5, 40], poison=False)
    o, lse, _, _ = tree_attention(c["q64"], c["k64"], c["v64"], c["vis"], c["lens"], c["trees"], 0.2)
    k, v = (np.repeat(c[n][1], 2, axis=1) for n in ("k64", "v64"))
    s = np.einsum("thd,nhd->thn", c["q64"][1], k) * 0.2
    see = np.ones((7, 40), dtype=bool)
    see[:, 33:] = c["vis"][1]
    s = np.where(see[:, None, :], s, -np.inf)
    p = np.exp(s)
    assert np.allclose(o[1], np.einsum("thn,nhd->thd", p, v) / p.sum(-1)[..., None], rtol=1e-12, atol=1e-13)
    assert np.allclose(lse[1], np.log(p.sum(-1)), rtol=1e-12)
    assert not o[0, :2].any() and np.isneginf(lse[0, :2]).all()   # 5 positions: nodes 0 and 1 are not in the cache


def test_a_chain_is_the_oracles_several_new_tokens():
    w = syn.make_contiguous(77, 2, 8, 2, 64, 60, [60, 33])
    w.q = syn.normal_bf16(78, (2, 6, 8, 64))
    f = lambda bits: torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double().numpy()  # noqa: E731
    k, v = f(w.k), f(w.v)
    vis = np.broadcast_to(np.tril(np.ones((6, 6), dtype=bool)), (2, 6, 6))
    o, lse, _, _ = tree_attention(f(w.q), [k[0], k[1, :33]], [v[0], v[1, :33]], vis, [60, 33], [6, 6], w.scale)
    ro, rl = oracle.attend(w)
    assert np.allclose(o, ro, rtol=1e-9, atol=1e-12) and np.allclose(lse, rl, rtol=1e-9)


def test_trees_and_masks():
    vis = tree_visibility([-1, 0, 0, 2, -1])
    assert vis.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]]
    rng = np.random.default_rng(0)
    vis = np.stack([tree_visibility(random_tree(rng, 130)) for _ in range(2)])
    words = pack_mask(vis)
    assert words.shape == (2, 130, 3)
    for b, i, j in ((0, 0, 0), (1, 129, 129), (1, 100, 64), (0, 65, 63), (0, 127, 1)):
        assert bool(int(words[b, i, j // 64]) >> (j % 64) & 1) == vis[b, i, j]


def test_tables_by_hand():
    table = np.array([[7, -1, -1], [3, 4, -1]])
    t, slots, cu, lens, held, left, bits = tables([3, 8], [2, 1], None, table, [10, 11, 12], 3, 4, 20, 5)
    assert t.tolist() == [[7, 12, -1], [3, 4, 11]] and slots.tolist() == [31, 48, 44, -1, -1]
    assert (cu, lens, held, left, bits) == ([0, 2, 3], [5, 9], [2, 3], 1, 0)
    assert tables([4], [4], None, np.array([[1, -1]]), [], 0, 4, 20, 4)[1].tolist() == [-1] * 4


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
def test_fp8_round_is_torchs(kv):
    t = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kv]
    x = torch.cat([torch.randn(20000) * 10.0 ** torch.linspace(-6, 2, 20000), torch.arange(0, 449, 0.5), torch.tensor([2.0 ** -10, 2.0 ** -17])])
    top = torch.finfo(t).max
    assert np.array_equal(fp8_round(x.numpy(), kv), x.clamp(-top, top).to(t).double().numpy())
