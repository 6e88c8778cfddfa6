"""Plain 64-bit forms of the 4-bit cache and of the window attention, and
inputs for their tests.  numpy and torch on the CPU only."""
import math

import numpy as np
import torch

from spec_util import TYPES, _bytes, _fill

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def round_e2m1_code(y):
    """E2M1 codes of fp32 y: the nearest value, ties to the even code, at most 6; the sign bit is y's."""
    a = np.abs(y.astype(np.float64))
    code = np.zeros(a.shape, dtype=np.uint8)
    for i in range(8):
        lo = (E2M1[i - 1] + E2M1[i]) / 2 if i else -1.0
        code[(a > lo) | ((a == lo) & (i % 2 == 0))] = i
    return code | (np.signbit(y).astype(np.uint8) << 3)


def e4m3_code(x):
    """E4M3 codes of fp32 x >= 0: nearest, ties to even, at most 448; NaN stays."""
    x = x.astype(np.float64)
    ok = np.isfinite(x)
    _, e = np.frexp(np.where(ok, x, 1.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3)
    v = np.minimum(np.round(np.where(ok, x, 1.0) / step) * step, 448.0)
    v = np.where(np.isposinf(x), 448.0, v)
    return np.where(np.isnan(x), 0x7F, torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()).astype(np.uint8)


def quantise4(x, t):
    """(codes uint8 [.., D / 2], scale codes uint8 [.., D / 16]) of 16-bit rows, by fd_cache_write4's definition in fp32."""
    x = x.float().numpy().reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    t = np.float32(t)
    with np.errstate(all="ignore"):
        s = e4m3_code(np.abs(x).max(-1) / (np.float32(6) * t))
        unit = torch.from_numpy(s).view(torch.float8_e4m3fn).float().numpy() * t
        use = unit > 0
        y = np.where(use[..., None], x / np.where(use, unit, 1)[..., None], np.float32(0))
    codes = round_e2m1_code(y).reshape(*x.shape[:-2], 16 * x.shape[-2])
    return codes[..., 0::2] | codes[..., 1::2] << 4, s


def values4(codes, scales, t=1.0):
    """fp64 values of codes [.., D / 2] and E4M3 scale codes [.., D / 16]."""
    grid = np.concatenate([E2M1, -E2M1])
    x = np.stack([grid[codes & 15], grid[codes >> 4]], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    s = torch.from_numpy(np.ascontiguousarray(scales)).view(torch.float8_e4m3fn).double().numpy()
    return x * np.repeat(s, 16, -1) * float(np.float32(t))


def sees(L, T, i, window, sinks):
    """Positions that new token i of T of a request of length L sees, as a bool array of L."""
    pos, p = np.arange(L), L - T + i
    v = pos <= p
    if window:
        v &= (pos < sinks) | (pos > p - window)
    return v


def attention(q, k, v, lens, window, sinks, scale, v_scale=1.0):
    """O, LSE, and per-element error bounds of an fp32 kernel, in 64 bits.

    q [B, T, Hq, D], k and v lists of [L_b, Hkv, D] (fp64, dequantised but for v_scale).

    The bounds, as for spec_util.tree_attention: a score is an fp32 dot product of D exact products,
    off by at most es = D 2^-23 scale sum|q k|.  A weight is then off relatively by 2 es, by the
    rounding of its argument (|s - m| 2^-23 and 2^-22 of the function), and by its parts: fp16 2^-10
    2^-11, bf16 2^-7 2^-7 2^-8; below 2^-20 together.  A weight in fp16 parts, 2^13 to 2^14 times itself
    for the largest, ends at half of fp16's least step, 2^-25: below 2^-38 of the largest it may be lost
    whole, of every V (allowed: 2^-37).  Sums over n positions in fp32 steps that may truncate: n 2^-23."""
    B, T, hq, D = q.shape
    G = hq // k[0].shape[1]
    o, lse = np.zeros((B, T, hq, D)), np.full((B, T, hq), -np.inf)
    eo, el = np.zeros((B, T, hq, D)), np.zeros((B, T, hq))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for b in range(B):
            for i in range(T):
                see = sees(lens[b], T, i, window, sinks)
                n = int(see.sum())
                if not n:
                    continue
                kk, vv = k[b][see].repeat(G, 1), v[b][see].repeat(G, 1)     # [n, hq, D]
                s = np.einsum("nhd,hd->hn", kk, q[b, i]) * scale
                es = D * 2.0 ** -23 * abs(scale) * np.einsum("nhd,hd->hn", np.abs(kk), np.abs(q[b, i])).max(-1)
                m = s.max(-1)
                p = np.exp(s - m[:, None])
                l = p.sum(-1)
                lse[b, i] = m + np.log(l)
                o[b, i] = np.einsum("hn,nhd->hd", p, vv) / l[:, None] * v_scale
                rel = 2 * es + 2.0 ** -20 + (m - s.min(-1)) * 2.0 ** -22 + (2 * n + 64) * 2.0 ** -23
                av = np.abs(vv)
                eo[b, i] = (2 * rel[:, None] * np.einsum("hn,nhd->hd", p, av) / l[:, None] + 2.0 ** -37 * av.sum(0)) * abs(v_scale)
                el[b, i] = 2 * rel + np.abs(lse[b, i]) * 2.0 ** -21
    return o, lse, eo, el


def make_case(seed, B, T, hq, hkv, D, lens, kv="bf16", dtype=None, page=0, window=0, sinks=0, spare=3, std=1.5, s_max=None):
    """CPU tensors of one call.  kv: bf16, f16, e4m3, e5m2 or e2m1 (q's type `dtype`: kv's own, or bf16).
    What no new token sees holds NaN, and the table entries of pages without a visible position are -7."""
    g = torch.Generator().manual_seed(seed)
    dtype = dtype or (kv if kv in ("bf16", "f16") else "bf16")
    fp4 = kv == "e2m1"
    q = (torch.randn(B, T, hq, D, generator=g) * std).to(TYPES[dtype])
    union = [np.any([sees(n, T, i, window, sinks) for i in range(T)], 0) if n else np.zeros(0, bool) for n in lens]
    rows, f64 = [], []     # per request: the tensors K.., V.. as lists of [L, hkv, width], and K, V in fp64
    for n in lens:
        parts, exact = [], []
        for _ in range(2):
            x = torch.randn(n, hkv, D, generator=g)
            if fp4:
                codes, s = quantise4(x.bfloat16(), 0.25)
                parts += [torch.from_numpy(codes), torch.from_numpy(s)]
                exact.append(values4(codes, s))
            else:
                x = x.to(TYPES[kv])
                parts.append(x)
                exact.append(x.float().numpy().astype(np.float64))
        rows.append(parts)
        f64.append(exact)
    nan = torch.tensor([0x7F], dtype=torch.uint8) if fp4 else torch.full((1,), math.nan).to(TYPES[kv])
    widths = [D // 2, D // 16] * 2 if fp4 else [D, D]
    s_max = s_max or max(max(lens), 1)
    if page:
        blocks = max(1, -(-max(lens) // page)) + 1
        live = [[bool(u[j * page:(j + 1) * page].any()) for j in range(blocks)] for u in union]
        pages = sum(map(sum, live)) + spare
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((B, blocks), -7, dtype=torch.int32)
        for b in range(B):
            for j in range(blocks):
                if live[b][j]:
                    table[b, j] = order.pop()
        place = lambda b, t: (int(table[b, t // page]), t % page)  # noqa: E731
    else:
        pages, page_rows, table = B, s_max, None
        place = lambda b, t: (b, t)  # noqa: E731
    page_rows = page or s_max
    pool = [_fill(nan, (pages, hkv, page_rows, w) if fp4 else (pages, page_rows, hkv, w)) for w in widths]
    for b, u in enumerate(union):
        at = np.nonzero(u)[0]
        if not len(at):
            continue
        where = np.array([place(b, int(t)) for t in at])
        pg, slot = torch.from_numpy(where[:, 0]), torch.from_numpy(where[:, 1])
        for t, x in zip(pool, rows[b]):
            y = _bytes(x)[torch.from_numpy(at)]
            if fp4:
                t[pg, :, slot] = y
            else:
                _bytes(t)[pg, slot] = y
    return dict(q=q, pool=pool, table=table, lens=list(lens), page=page, window=window, sinks=sinks, kv=kv, D=D, rows=rows,
                q64=q.float().numpy().astype(np.float64), k64=[x[0] for x in f64], v64=[x[1] for x in f64], place=place)


def want(c, scale, ks=1.0, vs=1.0):
    return attention(c["q64"], c["k64"], c["v64"], c["lens"], c["window"], c["sinks"], scale * ks, vs)


def run(fd, c, scale, **kw):
    """The library's call for a case."""
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    q, pool = c["q"].cuda(), [t.cuda() for t in c["pool"]]
    if c["kv"] == "e2m1":
        args, cache = dict(window=c["window"], sinks=c["sinks"], scale=scale, **kw), fd.Cache4(*pool)
        if c["page"]:
            return fd.fd_decode4_paged(q, cache, c["table"].cuda(), lens, **args)
        return fd.fd_decode4(q, cache, lens, **args)
    args = (lens, c["window"] or 2 ** 31 - 1, c["sinks"])
    if c["page"]:
        return fd.fd_window_decode_paged(q, *pool, c["table"].cuda(), *args, scale=scale, **kw)
    return fd.fd_window_decode(q, *pool, *args, scale=scale, **kw)
