"""The four calls together, as a speculative decoding loop uses them: pages
for the drafted tokens, their rows into the cache, the tree's attention, the
accepted path kept, over several steps -- against a cache kept in plain lists."""
import numpy as np
import pytest
import torch

from spec_util import TYPES, check_tree, fp8_quantise, pack_mask, random_tree, tree_attention, tree_visibility

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv,page", [("same", 16), ("same", 64), ("e4m3", 16), ("same", 4)])
def test_loop(fd, kv, page):
    rng = np.random.default_rng(page)
    B, T, hq, hkv, D, pages, steps, ma = 4, 12, 8, 2, 128, 200, 4, 5
    ks, vs = (0.03, 0.02) if kv != "same" else (1.0, 1.0)
    kt = TYPES["bf16" if kv == "same" else kv]
    pool_k, pool_v = (torch.full((pages, page, hkv, D), float("nan"), device="cuda").to(kt) for _ in range(2))
    table = torch.full((B, 1024 // page), -1, dtype=torch.int32, device="cuda")
    free, free_count = i32(rng.permutation(pages).tolist()), i32([pages])
    lens, held = i32([0] * B), i32([0] * B)
    ref = [[np.zeros((0, hkv, D))] * 2 for _ in range(B)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = fd.make_tree_workspace(B, T, hq, hkv, D)
    value = (lambda x, s: x.double().cpu().numpy()) if kv == "same" else (lambda x, s: fp8_quantise(x, s, kv))

    def append(new):
        nonlocal lens, held, free_count
        total = sum(new)
        t = fd.fd_build_tables(lens, i32(new), table, free, free_count, page, pages, total + 3, held_pages=held,
                               device_status=status)
        lens, held, free_count = t.seq_lens, t.held_pages, t.free_count
        qkv = (torch.randn(total + 3, (hq + 2 * hkv) * D, device="cuda") * 1.5).to(torch.bfloat16)
        k, v = (qkv[:, (hq + i * hkv) * D:(hq + (i + 1) * hkv) * D].unflatten(1, (hkv, D)) for i in range(2))
        fd.fd_cache_write(k, v, t.slot_map, pool_k, pool_v, k_scale=ks, v_scale=vs, device_status=status)
        at = 0
        for b in range(B):
            for i, (x, s) in enumerate(((k, ks), (v, vs))):
                ref[b][i] = np.concatenate([ref[b][i], value(x[at:at + new[b]], s)])
            at += new[b]

    append([5, 200, 1, 77])                      # prompts
    for _ in range(steps):
        append([T] * B)                          # drafted tokens
        trees = [random_tree(rng, T) for _ in range(B)]
        vis = np.stack([tree_visibility(p) for p in trees])
        q = torch.randn(B, T, hq, D, device="cuda").to(torch.bfloat16)
        o, l = fd.fd_tree_decode_paged(q, pool_k, pool_v, table, lens, torch.from_numpy(pack_mask(vis).view(np.int64)).cuda(),
                                       scale=0.1, k_scale=ks, v_scale=vs, workspace=ws)
        n = [len(ref[b][0]) for b in range(B)]
        assert lens.tolist() == n
        check_tree(o, l, tree_attention(q.double().cpu().numpy(), [r[0] for r in ref], [r[1] for r in ref], vis, n, [T] * B,
                                        0.1 * ks, vs))
        paths = []
        for p in trees:                          # the accepted path: a random node's ancestors
            node, path = int(rng.integers(0, T)), []
            while node >= 0:
                path.append(node)
                node = p[node]
            paths.append(path[::-1][:ma])
        lens = fd.fd_cache_compact(pool_k, pool_v, lens, i32([p + [0] * (ma - len(p)) for p in paths]), i32([len(p) for p in paths]),
                                   T, block_table=table, device_status=status)
        for b, p in enumerate(paths):
            for i in range(2):
                base = len(ref[b][i]) - T
                ref[b][i] = np.concatenate([ref[b][i][:base], ref[b][i][[base + x for x in p]]])
    assert int(status) == 0 and fd.fd_get_device_error(ws) == fd.FD_OK
    assert int(free_count) == pages - sum(held.tolist())   # no page was lost
