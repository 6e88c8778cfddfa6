"""Plain 64-bit forms of the speculative-decoding operators, and inputs for
their tests.  numpy and torch on the CPU only."""
import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def tables(old, new, held, table, free, count, page, num_pages, max_tokens):
    """fd_build_tables by its definition, on lists and numpy arrays; also the status bits."""
    B, blocks = table.shape
    cap = blocks * page
    table, bits = table.copy(), 0
    cu, lens, held_out, slots = [0], [], [], []
    if not 0 <= count <= len(free):
        bits |= 2
    left = min(max(count, 0), len(free))
    for b in range(B):
        o = min(max(old[b], 0), cap)
        n = min(max(new[b], 0), cap - o)
        least = -(-o // page)
        h = least if held is None else held[b]
        hc = min(max(h, least), blocks)
        if (o, n, hc) != (old[b], new[b], h):
            bits |= 2
        if cu[-1] + n > max_tokens:
            bits |= 2
            n = max_tokens - cu[-1]
        need = max(0, -(-(o + n) // page) - hc)
        got = 0
        for j in range(need):
            if left:
                left -= 1
                got += 1
                if not 0 <= free[left] < num_pages:
                    bits |= 8
                table[b, hc + j] = free[left]
            else:
                bits |= 4
                table[b, hc + j] = -1
        for pos in range(o, o + n):
            pg = int(table[b, pos // page])
            ok = 0 <= pg < num_pages
            if not ok and pos // page < hc + got:
                bits |= 8
            slots.append(pg * page + pos % page if ok else -1)
        cu.append(cu[-1] + n)
        lens.append(o + n if got == need else min(o + n, (hc + got) * page))
        held_out.append(hc + got)
    slots += [-1] * (max_tokens - len(slots))
    return table, np.array(slots, dtype=np.int64), cu, lens, held_out, left, bits


def fp8_round(x, kv):
    """fp64 x to the nearest value of the FP8 type, ties to even, saturating; NaN stays."""
    mant, low, top = (3, -6, 448.0) if kv == "e4m3" else (2, -14, 57344.0)
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 1.0))
    step = np.exp2(np.maximum(e - 1, low) - mant)
    y = np.where(np.isfinite(x), np.round(x / step) * step, x)
    return np.where(np.isnan(x), np.nan, np.clip(y, -top, top))


def fp8_quantise(x, scale, kv):
    """The values that fd_cache_write stores for 16-bit x: the fp32 quotient x / scale (numpy's fp32
    division rounds to nearest, and x and scale are fp32 numbers) rounded to the FP8 type.  The
    quotient's own rounding matters next to a tie: 1.5 / fp32(0.03) = 50.0000011 is 50 in fp32 (a step
    there is 3.8e-6), halfway between the codes of 48 and 52."""
    with np.errstate(invalid="ignore"):
        return fp8_round(x.float().cpu().numpy() / np.float32(scale), kv)


def random_tree(rng, n):
    """Parents of n nodes: each hangs under an earlier node or under the context (-1)."""
    return [int(rng.integers(max(-1, i - 4), i)) for i in range(n)]


def tree_visibility(parents):
    n = len(parents)
    vis = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            vis[i] = vis[p]
        vis[i, i] = True
    return vis


def pack_mask(vis):
    """bool [..., T, T] to uint64 words [..., T, ceil(T / 64)]."""
    T = vis.shape[-1]
    words = -(-T // 64)
    full = np.zeros(vis.shape[:-1] + (64 * words,), dtype=np.uint64)
    full[..., :T] = vis
    full = full.reshape(vis.shape[:-1] + (words, 64))
    return (full << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)


def tree_attention(q, k, v, vis, lens, trees, scale, v_scale=1.0):
    """O, LSE, and per-element error bounds of an fp32 kernel, in 64 bits.

    q [B, T, Hq, D], k and v lists of [L_b, Hkv, D] (fp64 arrays, dequantised
    except v_scale), vis bool [B, T, T], lens and trees lists.

    The bounds: a score is an fp32 dot product of D exact products, off by at
    most es = D 2^-23 scale sum|q k| (2^-23: a step of an addition that may
    truncate).  A weight exp(s - m) is then off relatively by 2 es, by the
    rounding of its argument (|s - m| 2^-23 and 2^-22 of the function) and,
    where it is taken in two bf16 parts, by 2^-8 2^-8.  Sums over n positions
    add n 2^-23 relatively to sum p |v|, twice (O and the normalising sum),
    and merging adds a few steps.  A weight in fp16 parts, 2^8 times itself,
    ends at half of fp16's least step, 2^-25: below 2^-33 of the row's largest
    weight it may be lost whole, which adds 2^-33 sum |v|."""
    B, T, hq, D = q.shape
    hkv = k[0].shape[1]
    G = hq // hkv
    o, lse = np.zeros((B, T, hq, D)), np.full((B, T, hq), -np.inf)
    eo, el = np.zeros((B, T, hq, D)), np.zeros((B, T, hq))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for b in range(B):
            L, t = lens[b], trees[b]
            for i in range(t):
                if L - t + i < 0:
                    continue
                see = np.ones(L, dtype=bool)
                for j in range(t):
                    if L - t + j >= 0:
                        see[L - t + j] = vis[b, i, j]
                if not see.any():
                    continue
                n = int(see.sum())
                for h in range(hq):
                    kk, vv = k[b][see, h // G], v[b][see, h // G]
                    s = kk @ q[b, i, h] * scale
                    es = D * 2.0 ** -23 * abs(scale) * (np.abs(kk) @ np.abs(q[b, i, h])).max()
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    lse[b, i, h] = m + np.log(l)
                    o[b, i, h] = p @ vv / l * v_scale
                    rel = 2 * es + 2.0 ** -16 + 2.0 ** -21 + (m - s[np.isfinite(s)].min()) * 2.0 ** -22 + (2 * n + 64) * 2.0 ** -23
                    eo[b, i, h] = (2 * rel * (p @ np.abs(vv) / l) + 2.0 ** -33 * np.abs(vv).sum(0)) * abs(v_scale)
                    el[b, i, h] = 2 * rel + abs(lse[b, i, h]) * 2.0 ** -21
    return o, lse, eo, el


def check_tree(got_o, got_lse, want):
    """Outputs against tree_attention's within its bounds; what is not finite has to be equal."""
    o, lse, eo, el = want
    for got, ref, err, name in ((got_o, o, eo, "O"), (got_lse, lse, el, "LSE")):
        if got is None:
            continue
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN places differ"
        inf = np.isinf(ref)
        assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), f"{name}: infinities differ"
        fin = np.isfinite(ref)
        off = np.abs(got[fin] - ref[fin])
        bad = off > err[fin]
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} outside the bound, worst {off.max():.3g} ({(off / np.maximum(err[fin], 1e-300)).max():.3g} of its bound)"


def make_tree_case(seed, B, T, hq, hkv, D, lens, trees=None, dtype="bf16", kv="same", page=0, s_max=None, spare=3,
                   poison=True, std=1.5):
    """CPU tensors of one call: q, cache (contiguous or pages, NaN where nothing may be read when
    poison), mask words, and the fp64 pieces that tree_attention takes."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    kvt = TYPES[dtype if kv == "same" else kv]
    trees = trees if trees is not None else [T] * B
    s_max = s_max or max(max(lens), 1)
    q = (torch.randn(B, T, hq, D, generator=g) * std).to(TYPES[dtype])
    k = [torch.randn(n, hkv, D, generator=g).to(kvt) for n in lens]
    v = [torch.randn(n, hkv, D, generator=g).to(kvt) for n in lens]
    vis = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        vis[b] = tree_visibility(random_tree(rng, T))
    nan = torch.full((1,), math.nan if poison else 0.0).to(kvt)
    if page:
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((B, max(1, max(need)) + 1), -7, dtype=torch.int32)
        pool = [_fill(nan, (pages, page, hkv, D)) for _ in range(2)]
        for b in range(B):
            for j in range(need[b]):
                pg = order.pop()
                table[b, j] = pg
                n = min(page, lens[b] - j * page)
                for t, x in zip(pool, (k[b], v[b])):
                    _bytes(t)[pg, :n] = _bytes(x)[j * page:j * page + n]
        extra = dict(block_table=table)
    else:
        pool = [_fill(nan, (B, s_max, hkv, D)) for _ in range(2)]
        for b in range(B):
            for t, x in zip(pool, (k[b], v[b])):
                _bytes(t)[b, :lens[b]] = _bytes(x)
        extra = {}
    f64 = lambda xs: [x.float().numpy().astype(np.float64) for x in xs]  # noqa: E731
    return dict(q=q, k=pool[0], v=pool[1], vis=vis, lens=list(lens), trees=list(trees), page=page,
                k64=f64(k), v64=f64(v), q64=q.float().numpy().astype(np.float64), **extra)


def _bytes(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16)


def _fill(value, shape):
    return _bytes(value).repeat(math.prod(shape)).view(shape).view(value.dtype)
