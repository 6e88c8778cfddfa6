"""fd_build_tables, fd_cache_write and fd_cache_compact on the GPU, against their definitions."""
import numpy as np
import pytest
import torch

from spec_util import TYPES, fp8_quantise, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- tables

def run_tables(fd, old, new, held, blocks, page, pages, free, count, max_tokens, seed=0):
    rng = np.random.default_rng(seed)
    B = len(old)
    table = rng.integers(0, pages, (B, blocks)).astype(np.int32)   # what held pages say; the rest must stay
    want = tables(old, new, held, table, free, count, page, pages, max_tokens)
    st = status()
    got = fd.fd_build_tables(i32(old), i32(new), torch.from_numpy(table).cuda(), i32(free), i32([count]), page, pages,
                             max_tokens, held_pages=None if held is None else i32(held), device_status=st)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), np.array(w).reshape(g.shape)), (g, w)
    assert int(st) == want[6]
    return want


@pytest.mark.parametrize("B,page,seed", [(1, 1, 0), (3, 16, 1), (64, 16, 2), (257, 7, 3), (1000, 128, 4), (4096, 2, 5)])
def test_tables_random(fd, B, page, seed):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, 5 * page + 2, B)
    new = rng.integers(0, 3 * page + 2, B) * (rng.random(B) < 0.8)   # some requests get nothing
    held = -(-old // page) + rng.integers(0, 3, B)
    total = int(np.maximum(0, -(-(old + new) // page) - held).sum())
    pages = total + 50
    free = rng.permutation(pages).tolist()
    for h in (None, held.tolist()):
        run_tables(fd, old.tolist(), new.tolist(), h, 12, page, pages, free, len(free), int(new.sum()) + 37, seed)


def test_tables_long_prompts_and_one_request(fd):
    run_tables(fd, [0, 5, 100000], [70000, 0, 1], None, 8000, 16, 9000, list(range(9000)), 9000, 70100)
    run_tables(fd, [0], [1], None, 1, 1, 1, [0], 1, 1)
    run_tables(fd, [4], [0], None, 4, 4, 8, [3, 1], 2, 0)   # no slot map at all


def test_tables_pages_run_out(fd):
    w = run_tables(fd, [15, 3, 32], [40, 2, 20], None, 8, 16, 64, [9, 8, 7], 3, 70)
    assert w[6] == 4 and w[5] == 0
    assert run_tables(fd, [0, 0], [1, 1], None, 4, 8, 8, [], 0, 4)[6] == 4
    assert run_tables(fd, [0, 8], [8, 8], [0, 3], 4, 8, 8, [5, 6, 7], 1, 16)[6] == 0


@pytest.mark.parametrize("old,new,held,free,count,tokens", [
    ([-3, 4], [2, 2], None, [0, 1, 2], 3, 8),          # negative length
    ([4, 4], [-2, 2], None, [0, 1, 2], 3, 8),          # negative new tokens
    ([30, 4], [10, 2], None, [0, 1, 2], 3, 40),        # past the table
    ([2 ** 31 - 1, 4], [2 ** 31 - 1, 2], None, [0, 1, 2], 3, 40),
    ([4, 4], [6, 6], None, [0, 1, 2, 3], 4, 9),        # past max_tokens
    ([9, 4], [1, 1], [1, 99], [0, 1, 2], 3, 8),        # held pages below the length, above the table
    ([4, 4], [6, 6], None, [0, 99, -5, 3], 4, 12),     # pages outside the pool
    ([4, 4], [6, 6], None, [0, 1, 2, 3], 9, 12),       # a count above the stack
    ([4, 4], [6, 6], None, [0, 1, 2, 3], -1, 12),
])
def test_tables_bad_device_values(fd, old, new, held, free, count, tokens):
    assert run_tables(fd, old, new, held, 4, 8, 16, free, count, tokens)[6] != 0


def test_tables_empty_batch_and_refusals(fd):
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    got = fd.fd_build_tables(z, z, torch.empty(0, 4, dtype=torch.int32, device="cuda"), i32([3]), i32([1]), 16, 8, 5)
    assert got.slot_map.tolist() == [-1] * 5 and got.cu_new_lens.tolist() == [0] and got.free_count.tolist() == [1]
    a = i32([1, 2])
    with pytest.raises(ValueError):
        fd.fd_build_tables(a, i32([1]), i32([[0], [0]]), a, i32([1]), 16, 8, 5)
    with pytest.raises(ValueError):
        fd.fd_build_tables(a.cpu(), a, i32([[0], [0]]), a, i32([1]), 16, 8, 5)
    with pytest.raises(ValueError):
        fd.fd_build_tables(a.long(), a, i32([[0], [0]]), a, i32([1]), 16, 8, 5)
    with pytest.raises(fd.FdError):
        fd.fd_build_tables(a, a, i32([[0], [0]]), a, i32([1]), 0, 8, 5)


# ---------------------------------------------------------------- write

def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8).cpu(), b.contiguous().view(torch.uint8).cpu())


@pytest.mark.parametrize("n,h,d,strided", [(1, 1, 64, False), (7, 8, 128, True), (300, 5, 64, True), (129, 32, 256, False),
                                           (1000, 2, 128, True), (33, 72, 128, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_write_16bit(fd, n, h, d, strided, dtype):
    g = torch.Generator(device="cuda").manual_seed(n)
    src = torch.randn(n, 3 * h * d, generator=g, device="cuda").to(TYPES[dtype])
    k, v = (src[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in (1, 2))
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(n + 50, generator=g, device="cuda")[:n]
    slots[::5] = -1
    ck, cv = (torch.randn(n + 50, h, d, generator=g, device="cuda").to(TYPES[dtype]) for _ in range(2))
    wk, wv = ck.cpu(), cv.cpu()
    keep = slots.cpu() >= 0
    wk[slots.cpu()[keep]], wv[slots.cpu()[keep]] = k.cpu()[keep], v.cpu()[keep]
    st = status()
    fd.fd_cache_write(k, v, slots, ck, cv, device_status=st)
    assert same_bytes(ck, wk) and same_bytes(cv, wv) and int(st) == 0


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,h,d", [(1, 1, 64), (77, 3, 128), (40, 8, 256)])
def test_write_fp8(fd, kv, dtype, n, h, d):
    """Codes equal the definition's: the nearest value of x / scale, ties to even, saturating, NaN kept."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = ((torch.randn(n, h, d, generator=g, device="cuda") * 10 ** (torch.rand(n, h, d, generator=g, device="cuda") * 8 - 4))
            .to(TYPES[dtype]) for _ in range(2))
    k.view(-1)[:10] = torch.tensor([float("inf"), -float("inf"), float("nan"), 448, 464, -480, 0.0, -0.0, 17, 19],
                                   device="cuda").to(k.dtype)   # 17, 19: ties of E4M3 (between 16, 18 and 20) at scale 1
    slots = torch.randperm(n + 9, generator=g, device="cuda")[:n]
    ck, cv = (torch.zeros(n + 9, h, d, device="cuda").to(TYPES[kv]) for _ in range(2))
    for ks, vs in ((1.0, 0.37), (0.03, 0.02), (1e-30, 2e30), (2.0 ** -60, 3.3e-7), (0.01234, 3.0)):
        fd.fd_cache_write(k, v, slots, ck, cv, k_scale=ks, v_scale=vs)
        for x, c, s in ((k, ck, ks), (v, cv, vs)):
            want = fp8_quantise(x, s, kv)
            got = c.view(torch.uint8)[slots].view(c.dtype).double().cpu().numpy()
            assert np.array_equal(got, want, equal_nan=True)
            num = ~np.isnan(want)
            assert np.array_equal(np.signbit(got[num]), np.signbit(want[num]))   # -0 stays -0
    # uint8 codes with kv_dtype are the same call
    c8, d8 = (torch.zeros(n + 9, h, d, device="cuda", dtype=torch.uint8) for _ in range(2))
    fd.fd_cache_write(k, v, slots, c8, d8, kv_dtype=kv, k_scale=0.01234, v_scale=3.0)
    assert torch.equal(c8[slots], ck.view(torch.uint8)[slots]) and torch.equal(d8[slots], cv.view(torch.uint8)[slots])


def test_write_bad_slots_and_refusals(fd):
    k = torch.randn(6, 2, 64, device="cuda", dtype=torch.bfloat16)
    ck, cv = (torch.zeros(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slots = torch.tensor([0, 8, 2 ** 40, -1, -2 ** 40, 7], device="cuda")
    st = status()
    fd.fd_cache_write(k, k, slots, ck, cv, device_status=st)
    assert int(st) == fd.FD_DEVICE_STATUS_BAD_SLOT
    flat = ck.view(8, 2, 64)
    assert torch.equal(flat[0], k[0]) and torch.equal(flat[7], k[5]) and not flat[1:7].any()
    with pytest.raises(TypeError):
        fd.fd_cache_write(k.half(), k.half(), slots, ck, cv)
    with pytest.raises(ValueError):
        fd.fd_cache_write(k, k, slots.int(), ck, cv)
    with pytest.raises(ValueError):
        fd.fd_cache_write(k.transpose(0, 1), k, slots, ck, cv)
    with pytest.raises(ValueError):
        fd.fd_cache_write(k[:, :1], k[:, :1], slots, ck, cv)
    with pytest.raises(fd.FdError):   # a token stride of 129 elements
        odd = torch.randn(6, 129, device="cuda", dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64))
        fd.fd_cache_write(odd, odd, slots, ck, cv)
    fd.fd_cache_write(k[:0], k[:0], slots[:0], ck, cv)


def test_write_past_32_bit_offsets(fd):
    """Rows whose byte offsets pass 2^32 (a 5 GB cache of each)."""
    h, d = 8, 128
    n = 5 * 2 ** 30 // (2 * h * d)
    ck, cv = (torch.zeros(n, h, d, device="cuda", dtype=torch.float16) for _ in range(2))
    k = torch.randn(3, h, d, device="cuda", dtype=torch.float16)
    slots = torch.tensor([n - 1, 2 ** 31 // (2 * h * d) + 1, 2 ** 32 // (2 * h * d) + 1], device="cuda")
    fd.fd_cache_write(k, -k, slots, ck, cv)
    assert torch.equal(ck[slots], k) and torch.equal(cv[slots], -k)
    assert int(ck.any(-1).any(-1).sum()) == 3


# ---------------------------------------------------------------- compact

def compact_case(seed, B, T, ma, h, d, page, kv, lens=None):
    rng = np.random.default_rng(seed)
    lens = lens or [int(x) for x in rng.integers(T, T + 3 * max(page, 8), B)]
    n = [int(x) for x in rng.integers(0, min(ma, T) + 1, B)]
    paths = [sorted(rng.choice(T, k, replace=False).tolist()) + [-9] * (ma - k) for k in n]
    g = torch.Generator().manual_seed(seed)
    if page:
        need = [-(-x // page) for x in lens]
        order = rng.permutation(sum(need) + 2).tolist()
        table = torch.full((B, max(need) + 1), -4, dtype=torch.int32)
        for b in range(B):
            for j in range(need[b]):
                table[b, j] = order.pop()
        shape = (sum(need) + 2, page, h, d)
    else:
        table, shape = None, (B, max(lens) + 2, h, d)
    k, v = (torch.randn(shape, generator=g).to(TYPES[kv]) for _ in range(2))
    return lens, n, paths, table, k, v


def plain_compact(k, v, lens, trees, n, paths, table):
    out = []
    for t in (k, v):
        y = t.clone().view(torch.uint8).view(-1, t.shape[2] * t.shape[3] * t.element_size())
        x, P = y.clone(), t.shape[1]
        row = lambda b, pos: int(table[b, pos // P]) * P + pos % P if table is not None else b * P + pos  # noqa: E731
        for b in range(len(lens)):
            for j in range(n[b]):
                y[row(b, lens[b] - trees[b] + j)] = x[row(b, lens[b] - trees[b] + paths[b][j])]
        out.append(y)
    return out


@pytest.mark.parametrize("page", [0, 1, 4, 16, 24, 64])
@pytest.mark.parametrize("B,T,ma,h,d,kv", [(1, 1, 1, 1, 64, "bf16"), (5, 64, 64, 8, 128, "bf16"), (3, 256, 256, 2, 64, "e4m3"),
                                           (2, 33, 9, 40, 256, "f16")])
def test_compact(fd, page, B, T, ma, h, d, kv):
    lens, n, paths, table, k, v = compact_case(page + B, B, T, ma, h, d, page, kv)
    n[-1] = min(ma, T)
    paths[-1] = (list(range(T - n[-1], T)) + [-9] * ma)[:ma]   # the longest path the arguments allow
    wk, wv = plain_compact(k, v, lens, [T] * B, n, paths, table)
    kd, vd, st = k.cuda(), v.cuda(), status()
    out = fd.fd_cache_compact(kd, vd, i32(lens), i32(paths), i32(n), T, block_table=None if table is None else table.cuda(),
                              device_status=st)
    assert out.tolist() == [L - T + x for L, x in zip(lens, n)] and int(st) == 0
    assert torch.equal(kd.view(torch.uint8).cpu().view(wk.shape), wk) and torch.equal(vd.view(torch.uint8).cpu().view(wv.shape), wv)


def test_compact_ragged_trees_and_identity(fd):
    lens, n, paths = [40, 12, 9, 0], [3, 2, 4, 0], [[0, 1, 2, -1], [1, 4, -1, -1], [0, 1, 2, 3], [-1] * 4]
    trees = [10, 5, 9, 0]
    k, v = (torch.randn(4, 40, 2, 64).to(torch.bfloat16) for _ in range(2))
    wk, wv = plain_compact(k, v, lens, trees, n, paths, None)
    kd, vd, st = k.cuda(), v.cuda(), status()
    out = fd.fd_cache_compact(kd, vd, i32(lens), i32(paths), i32(n), 10, tree_lens=i32(trees), device_status=st)
    assert out.tolist() == [33, 9, 4, 0] and int(st) == 0
    assert torch.equal(kd.view(torch.uint8).cpu().view(wk.shape), wk) and torch.equal(vd.view(torch.uint8).cpu().view(wv.shape), wv)


@pytest.mark.parametrize("lens,n,path,kept,bits", [
    ([20], [3], [4, 2, 5, 0], 1, 8),         # not ascending
    ([20], [3], [4, 4, 5, 0], 1, 8),         # twice the same node
    ([20], [2], [3, 8, 0, 0], 1, 8),         # outside the tree
    ([20], [2], [-1, 3, 0, 0], 0, 8),
    ([20], [9], [0, 2, 4, 6], 4, 2),         # more than the path holds
    ([20], [-5], [0, 2, 4, 6], 0, 2),
    ([5], [4], [0, 2, 3, 4], 4, 2),          # fewer tokens than drafted: the tree is cut to them
    ([-3], [0], [0, 0, 0, 0], 0, 2),
    ([99], [1], [1, 0, 0, 0], 1, 2),         # past the cache
])
def test_compact_bad_device_values(fd, lens, n, path, kept, bits):
    k, v = (torch.randn(1, 24, 2, 64).to(torch.bfloat16) for _ in range(2))
    L = min(max(lens[0], 0), 24)
    t = min(8, L)
    wk, wv = plain_compact(k, v, [L], [t], [kept], [path], None)
    kd, vd, st = k.cuda(), v.cuda(), status()
    out = fd.fd_cache_compact(kd, vd, i32(lens), i32([path]), i32(n), 8, device_status=st)
    assert out.tolist() == [L - t + kept] and int(st) == bits
    assert torch.equal(kd.view(torch.uint8).cpu().view(wk.shape), wk) and torch.equal(vd.view(torch.uint8).cpu().view(wv.shape), wv)


def test_compact_bad_pages_and_refusals(fd):
    k, v = (torch.randn(3, 4, 2, 64).to(torch.bfloat16) for _ in range(2))
    for table, kept in (([[0, 1, 9]], 1), ([[0, -1, 2]], 1), ([[0, 1, 2]], 2)):
        kd, vd, st = k.cuda(), v.cuda(), status()
        # base 4, nodes at 4 .. 11: node 1 (position 5, page 1), node 6 (position 10, page 2)
        out = fd.fd_cache_compact(kd, vd, i32([12]), i32([[1, 6]]), i32([2]), 8, block_table=i32(table), device_status=st)
        ok = 2 if kept == 2 else (1 if table[0][1] == 1 else 0)
        assert out.tolist() == [4 + ok] and int(st) == (0 if ok == 2 else 8)
    with pytest.raises(ValueError):
        fd.fd_cache_compact(k.cuda(), v.cuda(), i32([4]), i32([[1]]), i32([1]), 4)
    with pytest.raises(fd.FdError):
        lens = i32([4, 4, 4])
        fd.fd_cache_compact(k.cuda(), v.cuda(), lens, i32([[1]] * 3), i32([1] * 3), 4, seq_lens_out=lens)
