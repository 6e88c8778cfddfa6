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


def state(kv, seed=0, B=3, T=9, hq=8, hkv=2, D=128, page=16, pages=64):
    """What a program keeps between steps, and one step over it: all four calls, into given buffers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    kt = TYPES["bf16" if kv == "same" else kv]
    s = dict(k=torch.randn(pages, page, hkv, D, generator=g, device="cuda").to(kt),
             v=torch.randn(pages, page, hkv, D, generator=g, device="cuda").to(kt),
             table=torch.full((B, 24), -1, dtype=torch.int32, device="cuda"), free=i32(rng.permutation(pages).tolist()),
             count=i32([pages]), lens=i32([0] * B), held=i32([0] * B), new=i32([100, 17, 260]),
             kv_new=torch.randn(B, T, 2 * hkv, D, generator=g, device="cuda").to(torch.bfloat16),
             prompt=torch.randn(377, 2 * hkv, D, generator=g, device="cuda").to(torch.bfloat16),
             q=torch.randn(B, T, hq, D, generator=g, device="cuda").to(torch.bfloat16),
             path=i32([[0, 3, 5], [1, 2, 8], [4, 0, 0]]), npath=i32([3, 2, 1]), status=i32([0]), T=T, page=page, pages=pages, hkv=hkv)
    vis = np.stack([tree_visibility(random_tree(rng, T)) for _ in range(B)])
    s["mask"] = torch.from_numpy(pack_mask(vis).view(np.int64)).cuda()
    return s


def step(fd, s, ws):
    """Append T drafted rows to every request, attend, keep a path; the state's lengths, pages and stack move on."""
    h, B = s["hkv"], s["lens"].shape[0]
    scales = dict(k_scale=0.02, v_scale=0.03) if s["k"].element_size() == 1 else {}
    t = fd.fd_build_tables(s["lens"], s["new"], s["table"], s["free"], s["count"], s["page"], s["pages"], B * s["T"],
                           held_pages=s["held"], device_status=s["status"])
    rows = s["kv_new"].view(B * s["T"], 2 * h, -1)
    fd.fd_cache_write(rows[:, :h], rows[:, h:], t.slot_map, s["k"], s["v"], device_status=s["status"], **scales)
    out, lse = fd.fd_tree_decode_paged(s["q"], s["k"], s["v"], s["table"], t.seq_lens, s["mask"], workspace=ws, **scales)
    lens = fd.fd_cache_compact(s["k"], s["v"], t.seq_lens, s["path"], s["npath"], s["T"], block_table=s["table"],
                               device_status=s["status"])
    for name, x in (("lens", lens), ("held", t.held_pages), ("count", t.free_count)):
        s[name].copy_(x)
    return out, lse


def prefill(fd, s):
    """The prompts, by the same calls."""
    h = s["hkv"]
    scales = dict(k_scale=0.02, v_scale=0.03) if s["k"].element_size() == 1 else {}
    t = fd.fd_build_tables(s["lens"], s["new"], s["table"], s["free"], s["count"], s["page"], s["pages"], 377,
                           held_pages=s["held"])
    fd.fd_cache_write(s["prompt"][:, :h], s["prompt"][:, h:], t.slot_map, s["k"], s["v"], **scales)
    for name, x in (("lens", t.seq_lens), ("held", t.held_pages), ("count", t.free_count)):
        s[name].copy_(x)
    s["new"].fill_(s["T"])


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_captured_step_replays_as_eager_steps(fd, kv):
    """A step captured once and replayed gives bit for bit what eager steps give, with new rows each time."""
    a, b = state(kv), state(kv)
    ws_a, ws_b = (fd.make_tree_workspace(3, 9, 8, 2) for _ in range(2))
    for s in (a, b):
        prefill(fd, s)
    eager = []
    for n in range(4):
        a["kv_new"].mul_(-1)
        a["q"].add_(0.25)
        out, lse = step(fd, a, ws_a)
        eager.append((out.clone(), lse.clone()))
    side = state(kv, seed=1)   # a first call of each shape outside the capture
    prefill(fd, side)
    step(fd, side, ws_b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(fd, b, ws_b)
    for n in range(4):
        b["kv_new"].mul_(-1)
        b["q"].add_(0.25)
        graph.replay()
        assert same(out, eager[n][0]) and same(lse, eager[n][1]), n
    for name in ("k", "v", "table", "lens", "held", "count", "status"):
        assert same(a[name], b[name]), name
    assert int(a["status"]) == 0


def test_two_graphs_share_a_workspace_in_order(fd):
    """Graphs of different shapes replayed in turn on one workspace (of the larger shape), and on other streams."""
    c = [dict(q=torch.randn(2, T, 8, 128, device="cuda").half(), k=torch.randn(2, 700, 2, 128, device="cuda").half(),
              lens=i32([700, 90])) for T in (5, 50)]
    ws = fd.make_tree_workspace(2, 50, 8, 2)
    want_ = [fd.fd_tree_decode(x["q"], x["k"], x["k"], x["lens"]) for x in c]
    graphs, outs = [], []
    for x in c:
        fd.fd_tree_decode(x["q"], x["k"], x["k"], x["lens"], workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fd.fd_tree_decode(x["q"], x["k"], x["k"], x["lens"], workspace=ws))
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want_):
        assert same(o, wo) and same(l, wl)


def test_concurrent_streams_with_their_own_workspaces(fd):
    q, k, lens = torch.randn(4, 20, 8, 128, device="cuda").half(), torch.randn(4, 3000, 2, 128, device="cuda").half(), i32([3000, 5, 777, 2000])
    want_ = fd.fd_tree_decode(q, k, k, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for n in range(12):   # each call's outputs and workspace belong to its stream
        got.append(fd.fd_tree_decode(q, k, k, lens, stream=streams[n % 3]))
    torch.cuda.synchronize()
    for o, l in got:
        assert same(o, want_[0]) and same(l, want_[1])
    with torch.cuda.stream(streams[0]):
        o, l = fd.fd_tree_decode(q, k, k, lens)
    streams[0].synchronize()
    assert same(o, want_[0])


def test_repeated_calls_are_bitwise_equal(fd):
    q = torch.randn(2, 40, 16, 128, device="cuda").to(torch.bfloat16)
    k = torch.randn(2, 9000, 2, 128, device="cuda").to(torch.bfloat16)
    lens = i32([9000, 6000])
    first = fd.fd_tree_decode(q, k, k, lens)
    for _ in range(20):
        o, l = fd.fd_tree_decode(q, k, k, lens)
        assert same(o, first[0]) and same(l, first[1])
