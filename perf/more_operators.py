"""Workloads of the 4-bit cache and of the sliding window with sinks, with their plain forms.

Four operators, which make a long context's cache stream shorter:

  write4   new K/V rows quantised into a 4-bit cache (and read back, as what the cache now stands for)
  read4    rows of a 4-bit cache as 16-bit rows
  decode4  decode attention over a 4-bit cache, whole or through a window
  window   decode attention through a sliding window with sinks, over a 16-bit or FP8 cache

A 4-bit cache holds E2M1 codes, two a byte (the even dim in the low half), and
an E4M3 scale for every 16 dims of a row, head by head inside a page: codes
[pages, Hkv, P, D / 2], scales [pages, Hkv, P, D / 16]; a contiguous cache is
[B, Hkv, S, ..].  An element is code * scale * (the call's k_scale or v_scale).

``run`` computes each in its plain form (elementary torch operations in fp32)
or, where ``own`` is set, with the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the rows of one decoding step of 64 requests: nothing but latency
        dict(name="write4_step", op="write4", tokens=64, slots=65536, kv_heads=8, dim=128, page=16, dtype="bf16",
             pad=0, strided=True),
        # a prefill wave's rows, cut out of a fused QKV projection, a padded end
        dict(name="write4_prefill", op="write4", tokens=32768, slots=65536, kv_heads=8, dim=128, page=64, dtype="bf16",
             pad=1000, strided=True),
        # a shared prefix handed to an attention over 16-bit rows
        dict(name="read4_prefix", op="read4", tokens=1500, slots=16384, kv_heads=8, dim=128, page=16, dtype="f16",
             pad=36),
        # the caches of a whole batch moved back into 16 bits
        dict(name="read4_batch", op="read4", tokens=98304, slots=131072, kv_heads=8, dim=128, page=64, dtype="bf16",
             pad=0),
        # one short request of a small MHA model: latency
        dict(name="decode4_short", op="decode4", batch=1, q_len=1, heads=32, kv_heads=32, dim=128, page=0,
             len_min=2048, len_max=2048, dtype="bf16", window=0, sinks=0),
        # one long context, MHA
        dict(name="decode4_long", op="decode4", batch=1, q_len=1, heads=32, kv_heads=32, dim=128, page=0,
             len_min=131072, len_max=131072, dtype="bf16", window=0, sinks=0),
        # a ragged serving batch over 16-token pages, GQA-4
        dict(name="decode4_paged", op="decode4", batch=64, q_len=1, heads=32, kv_heads=8, dim=128, page=16,
             len_min=1, len_max=16384, dtype="bf16", window=0, sinks=0),
        # GQA-8 with two new tokens a request (16 query columns a kv head), fp16 queries
        dict(name="decode4_two_tokens", op="decode4", batch=8, q_len=2, heads=64, kv_heads=8, dim=128, page=64,
             len_min=4096, len_max=65536, dtype="f16", window=0, sinks=0),
        # one request through a short window: latency
        dict(name="window_short", op="window", batch=1, q_len=1, heads=32, kv_heads=8, dim=128, page=0,
             len_min=8000, len_max=8000, dtype="bf16", kv="same", window=1024, sinks=4),
        # long contexts whose pages behind the window were given back, GQA-4 over 16-token pages
        dict(name="window_paged", op="window", batch=64, q_len=1, heads=32, kv_heads=8, dim=128, page=16,
             len_min=64, len_max=131072, dtype="bf16", kv="same", window=4096, sinks=4),
        # GQA-8 over an FP8 cache
        dict(name="window_e4m3", op="window", batch=128, q_len=1, heads=64, kv_heads=8, dim=128, page=64,
             len_min=1024, len_max=65536, dtype="bf16", kv="e4m3", window=8191, sinks=4),
        # a check of four draft tokens, 64-dim heads, odd sizes, a contiguous fp16 cache
        dict(name="window_drafts", op="window", batch=29, q_len=4, heads=24, kv_heads=8, dim=64, page=0,
             len_min=1, len_max=4001, dtype="f16", kv="same", window=1537, sinks=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["write4", "read4", "decode4", "decode4", "decode4", "window", "window", "window"])
    if op in ("write4", "read4"):
        tokens = _log_int(rng, 1, 98304)
        page = rng.choice([1, 4, 16, 24, 64, 128])
        slots = -(-(tokens + _log_int(rng, 1, 65536)) // page) * page
        c = dict(op=op, tokens=tokens, slots=slots, kv_heads=rng.choice([1, 2, 5, 8, 32]),
                 dim=rng.choice([64, 128, 256]), page=page, dtype=rng.choice(["bf16", "f16"]), pad=rng.randint(0, 300))
        if op == "write4":
            c["strided"] = rng.random() < 0.5
        return c
    kv_heads, group, q_len = rng.choice([(32, 1, 1), (8, 1, 4), (8, 4, 1), (8, 8, 2), (4, 3, 5), (1, 16, 1), (2, 7, 2),
                                         (5, 2, 3), (16, 1, 16)])
    lo = _log_int(rng, 1, 8192)
    c = dict(op=op, batch=_log_int(rng, 1, 96), q_len=q_len, heads=kv_heads * group, kv_heads=kv_heads,
             dim=rng.choice([64, 128, 128, 256]), page=rng.choice([0, 0, 1, 4, 16, 64, 128]), len_min=lo,
             len_max=lo + _log_int(rng, 1, 65536), dtype=rng.choice(["bf16", "f16"]))
    c["window"] = _log_int(rng, 1, 16384)
    c["sinks"] = rng.choice([0, 0, 1, 4, 100])
    if op == "decode4":
        if rng.random() < 0.6:
            c["window"] = c["sinks"] = 0
    else:
        c["kv"] = rng.choice(["same", "same", "e4m3", "e5m2"])
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in m:
            m[k] = max(m[k], w[k])
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] > most[c["op"]]["bytes"] or w["flops"] > most[c["op"]]["flops"]:
            continue
        if c["op"] in ("decode4", "window"):
            # a contiguous cache is held whole, and the plain form's fp32 copies and scores stay within the card
            if not c["page"] and c["batch"] * c["len_max"] * c["kv_heads"] * c["dim"] > 3e9:
                continue
            if c["batch"] * _span(c, c["len_max"]) * (c["kv_heads"] * c["dim"] * 8 + c["heads"] * c["q_len"] * 16) > 60e9:
                continue
        return c


# ---------------------------------------------------------------- inputs

def _grid(lo, hi, n):
    """n whole numbers spread evenly from lo to hi (one: hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _first(case, n):
    """The first position behind the sinks that some new token of a request of length n sees."""
    if not case["window"]:
        return 0
    return min(n, max(case["sinks"], n - case["q_len"] - case["window"] + 1, 0))


def _span(case, n):
    """Positions that some new token of a request of length n sees."""
    first = _first(case, n)
    return n - first + min(case["sinks"], first)


def _rows(gen, shape, dtype, std=1.0):
    if math.prod(shape) < (1 << 26):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).to(dtype)


def _cache4(gen, pages, kv_heads, page, dim, scale):
    """Codes and block scales of a 4-bit cache that holds Gaussian rows."""
    codes = torch.empty(pages, kv_heads, page, dim // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, kv_heads, page, dim // 16, dtype=torch.uint8, device="cuda")
    c, s = codes.view(-1, dim // 2), scales.view(-1, dim // 16)
    n, step = c.shape[0], max(1, (1 << 26) // dim)
    for i in range(0, n, step):
        m = min(step, n - i)
        c[i:i + m], s[i:i + m] = _quantise4(torch.randn(m, dim, generator=gen, device="cuda"), scale)
    return codes, scales.view(torch.float8_e4m3fn)


def _paged(gen, lens, firsts, sinks, page, spare):
    """(block table, pages): the pages of positions [0, sinks) and [first, len) of every request, scattered over
    a pool with spare pages; the entries of all other pages are -1."""
    width = max(1, -(-max(lens) // page))
    j = torch.arange(width, device="cuda")[None, :]
    n = torch.tensor(lens, device="cuda")[:, None]
    first = torch.tensor(firsts, device="cuda")[:, None]
    live = (j * page < n) & ((j * page < sinks) | ((j + 1) * page > first))
    held = int(live.sum())
    pages = held + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full(live.shape, -1, dtype=torch.int32, device="cuda")
    table[live] = order[:held]
    return table, pages


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, H, D, P = case["op"], case["kv_heads"], case["dim"], case["page"]
    s = dict(case=dict(case))
    if op in ("write4", "read4"):
        n, pages = case["tokens"], case["slots"] // P
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int64)
        if case["pad"]:   # the padded end of a captured batch
            slots[max(1, n - case["pad"]):] = -1
        s.update(slots=slots, k_scale=0.01 * (1 + rng.random()), v_scale=0.01 * (1 + rng.random()))
        s["k"], s["v"] = (_cache4(gen, pages, H, P, D, s[x]) for x in ("k_scale", "v_scale"))
        if op == "write4":
            dt = _T[case["dtype"]]
            if case["strided"]:   # K and V as the last columns of a fused GQA-4 projection's output
                qkv = _rows(gen, (n, 6 * H * D), dt, 1.5)
                s["k_new"], s["v_new"] = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (4, 5))
            else:
                s["k_new"], s["v_new"] = (_rows(gen, (n, H, D), dt, 1.5) for _ in range(2))
        # where the rows come back to: the padded rows stay as they are
        s["k_out"], s["v_out"] = (torch.zeros(n, H, D, dtype=_T[case["dtype"]], device="cuda") for _ in range(2))
        return s
    B = case["batch"]
    lens = _grid(case["len_min"], case["len_max"], B)
    rng.shuffle(lens)
    if P:
        firsts = [_first(case, n) for n in lens]
        s["table"], pages = _paged(gen, lens, firsts, case["sinks"] if case["window"] else 0, P, 8)
        rows = P
    else:
        pages, rows = B, case["len_max"]
    s.update(q=_rows(gen, (B, case["q_len"], case["heads"], D), _T[case["dtype"]], 2.0), scale=1.0 / math.sqrt(D),
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if op == "decode4":
        s["k_scale"], s["v_scale"] = 0.01 * (1 + rng.random()), 0.01 * (1 + rng.random())
        s["k"], s["v"] = (_cache4(gen, pages, H, rows, D, s[x]) for x in ("k_scale", "v_scale"))
    else:
        kv = case["dtype"] if case["kv"] == "same" else case["kv"]
        s["k_scale"], s["v_scale"] = (1.0, 1.0) if case["kv"] == "same" else (0.5, 1.5)
        s["k"], s["v"] = (_rows(gen, (pages, rows, H, D), _T[kv]) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms

def _quantise4(x, scale):
    """(codes uint8 [.., D / 2], scale codes uint8 [.., D / 16]) of fp32 rows [.., D]."""
    x = x.unflatten(-1, (-1, 16))
    t = torch.tensor(scale, dtype=torch.float32, device=x.device)
    block = (x.abs().amax(-1) / (6 * t)).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = (block.float() * t)[..., None]
    y = torch.where(unit > 0, x / unit, torch.zeros_like(x))
    a = y.abs()
    # the number of values of E2M1 that a is nearer to than to 0: ties go to the even code
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], block.view(torch.uint8)


def _values4(codes, scales, scale):
    """fp32 values [.., D] of codes [.., D / 2] and E4M3 block scales [.., D / 16]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    pair = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    t = torch.tensor(scale, dtype=torch.float32, device=codes.device)
    return ((pair.unflatten(-1, (-1, 16)) * scales.float()[..., None]) * t).flatten(-2)


def _rows4(case, slots):
    """Rows [n, Hkv] of the codes and scales, flat over (page, head, token), of the slots."""
    H, P = case["kv_heads"], case["page"]
    return (slots // P)[:, None] * (H * P) + torch.arange(H, device="cuda")[None, :] * P + (slots % P)[:, None]


def _plain_read4(s):
    c = s["case"]
    ok = s["slots"] >= 0
    at = _rows4(c, s["slots"][ok])
    for (codes, scales), scale, out in ((s["k"], s["k_scale"], s["k_out"]), (s["v"], s["v_scale"], s["v_out"])):
        rows = scales.view(torch.uint8).view(-1, c["dim"] // 16)[at].view(torch.float8_e4m3fn)
        out[ok] = _values4(codes.view(-1, c["dim"] // 2)[at], rows, scale).to(out.dtype)
    return s["k_out"], s["v_out"]


def _plain_write4(s):
    c = s["case"]
    ok = s["slots"] >= 0
    at = _rows4(c, s["slots"][ok])
    for new, (codes, scales), scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        x, b = _quantise4(new[ok].float(), scale)
        codes.view(-1, c["dim"] // 2)[at] = x
        scales.view(torch.uint8).view(-1, c["dim"] // 16)[at] = b
    return (*_plain_read4(s), s["k"][1], s["v"][1])


def _plain_attention(s):
    c = s["case"]
    B, T, H, D, P = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["page"]
    G, window = c["heads"] // H, c["window"]
    sinks = c["sinks"] if window else 0
    lens = s["lens"].long()[:, None]
    # the positions that a request's new tokens see together, one after another, then masked ones
    first = torch.minimum(lens, (lens - T - window + 1).clamp(min=sinks)) if window else torch.zeros_like(lens)
    head = first.clamp(max=sinks)
    n = max(1, _span(c, c["len_max"]))   # a longer request's tokens see no fewer positions
    j = torch.arange(n, device="cuda")[None, :]
    pos = torch.where(j < head, j, j - head + first)
    live = pos < lens
    at = pos.clamp(max=c["len_max"] - 1)
    if P:
        page = torch.gather(s["table"], 1, at // P).long().clamp(min=0)
        slot = at % P
    else:
        page = torch.arange(B, device="cuda")[:, None].expand(B, n)
        slot = at

    def rows(x, scale):   # [B, H, n, D] fp32
        if c["op"] == "window":
            x = x.view(torch.uint8)[page, slot].view(x.dtype) if x.element_size() == 1 else x[page, slot]
            return x.float().transpose(1, 2)
        codes, scales = x
        h = torch.arange(H, device="cuda")[None, :, None]
        page4, slot4 = page[:, None, :], slot[:, None, :]
        return _values4(codes[page4, h, slot4], scales.view(torch.uint8)[page4, h, slot4].view(torch.float8_e4m3fn), scale)

    own_pos = lens - T + torch.arange(T, device="cuda")[None, :]          # [B, T]
    sees = (pos[:, None, :] <= own_pos[:, :, None]) & live[:, None, :]
    if window:
        sees &= (pos[:, None, :] < sinks) | (pos[:, None, :] > own_pos[:, :, None] - window)
    sees = sees[:, None, :, None, :]                                       # [B, 1, T, 1, n]
    k_scale, v_scale = (s["k_scale"], s["v_scale"]) if c["op"] == "window" else (1.0, 1.0)
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    x = torch.matmul(q, rows(s["k"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"] * k_scale).view(B, H, T, G, n)
    x = x.masked_fill_(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = x.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, T * G, n), rows(s["v"], s["v_scale"])).view(B, H, T, G, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-38) * v_scale, torch.zeros_like(o))
    lse = (m0 + total.log()).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D), lse.permute(0, 2, 1, 3).reshape(B, T, H * G))


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"write4": _plain_write4, "read4": _plain_read4, "decode4": _plain_attention, "window": _plain_attention}[c["op"]](s)
    import decode_attention_decoding_gb300 as fd
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "window":
        cache = (s["k"], s["v"])
    else:
        if "cache" not in s:   # a program keeps its cache's tensors together
            s["cache"] = fd.Cache4(s["k"][0], s["k"][1], s["v"][0], s["v"][1])
        cache = (s["cache"],)
    if c["op"] in ("write4", "read4"):
        if c["op"] == "write4":
            fd.fd_cache_write4(s["k_new"], s["v_new"], s["slots"], *cache, **scales)
        k, v = fd.fd_cache_read4(s["slots"], *cache, k_out=s["k_out"], v_out=s["v_out"], **scales)
        return (k, v, s["k"][1], s["v"][1]) if c["op"] == "write4" else (k, v)
    if "workspace" not in s:   # a program keeps one workspace for its calls
        s["workspace"] = fd.make_window_workspace(c["batch"], c["heads"], c["kv_heads"], c["dim"], q_len=c["q_len"])
    more = dict(scale=s["scale"], workspace=s["workspace"], **scales)
    if c["op"] == "decode4":
        more.update(window=c["window"], sinks=c["sinks"])
        if c["page"]:
            return fd.fd_decode4_paged(s["q"], *cache, s["table"], s["lens"], **more)
        return fd.fd_decode4(s["q"], *cache, s["lens"], **more)
    if c["page"]:
        return fd.fd_window_decode_paged(s["q"], *cache, s["table"], s["lens"], c["window"], c["sinks"], **more)
    return fd.fd_window_decode(s["q"], *cache, s["lens"], c["window"], c["sinks"], **more)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, D = case["kv_heads"], case["dim"]
    if case["op"] in ("write4", "read4"):
        n = max(min(case["tokens"], 1), case["tokens"] - case["pad"])
        wide, narrow = 2 * n * H * D * 2, 2 * n * H * (D // 2 + D // 16)
        # the rows once in 16 bits and once in 4; what was written comes back too
        twice = 2 if case["op"] == "write4" else 1
        return {"bytes": twice * (wide + narrow) + 8 * case["tokens"], "flops": 2 * twice * 2 * n * H * D}
    B, T, hq = case["batch"], case["q_len"], case["heads"]
    spans = sum(_span(case, n) for n in _grid(case["len_min"], case["len_max"], B))
    if case["op"] == "decode4":
        row = D // 2 + D // 16
    else:
        row = D * (2 if case["kv"] == "same" else 1)
    entries = spans // case["page"] + 2 * B if case["page"] else 0
    return {"bytes": 2 * row * H * spans + 6 * B * T * hq * D + 4 * B * T * hq + 4 * entries + 4 * B,
            "flops": 4 * hq * T * D * spans}


# ---------------------------------------------------------------- the definition in 64 bits

def _round4(x):
    """x (fp64) rounded to the nearest E2M1 value, ties to the even code, saturating."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.sign(x) * torch.clamp(torch.round(a / step) * step, max=6.0)   # torch.round: half to even


def _round_e4m3(x):
    """x >= 0 (fp64) rounded to the nearest E4M3 value, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = torch.exp2((torch.clamp(e - 1, min=-6) - 3).double())
    return torch.clamp(torch.round(x / step) * step, max=448.0)


def _exact_values4(cache, scale, rows):
    """fp64 values of flat rows of a 4-bit cache."""
    codes, scales = cache
    D = codes.shape[-1] * 2
    c = codes.view(-1, D // 2).index_select(0, rows)
    e = scales.view(torch.uint8).view(-1, D // 16).index_select(0, rows).view(torch.float8_e4m3fn).double()
    lo, hi = c.bitwise_and(15).long(), c.bitwise_right_shift(4).long()
    grid = torch.tensor([*_E2M1, *(-v for v in _E2M1)], dtype=torch.float64, device="cuda")
    x = torch.empty(c.shape[0], D, dtype=torch.float64, device="cuda")
    x[:, 0::2], x[:, 1::2] = grid[lo], grid[hi]
    return x * e.repeat_interleave(16, dim=1) * float(np.float32(scale))


def exact(case, seed):
    s = prepare(case, seed)
    op, H, D, P = case["op"], case["kv_heads"], case["dim"], case["page"]
    if op in ("write4", "read4"):
        live = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        slots = s["slots"].tolist()
        at = torch.tensor([(slots[i] // P * H + h) * P + slots[i] % P for i in live for h in range(H)], device="cuda")
        which = torch.tensor(live, device="cuda")
        values, scales = [], []
        for x in ("k", "v"):
            t = float(np.float32(s[x + "_scale"]))
            y = torch.zeros(case["tokens"], H, D, dtype=torch.float64, device="cuda")
            if op == "write4":
                new = s[x + "_new"].index_select(0, which).double().reshape(-1, D // 16, 16)
                b = _round_e4m3(new.abs().amax(-1) / (6 * t))
                unit = torch.where(b > 0, b * t, torch.ones_like(b))[..., None]
                got = torch.where(b[..., None] > 0, _round4(new / unit) * unit, torch.zeros_like(new)).view(-1, H, D)
                after = s[x][1].double().view(-1, D // 16)
                after.index_copy_(0, at, b.view(-1, D // 16))
                scales.append(after.view(s[x][1].shape))
            else:
                got = _exact_values4(s[x], s[x + "_scale"], at).view(-1, H, D)
            y.index_copy_(0, which, got)
            values.append(y)
        return (*values, *scales)
    B, T, G = case["batch"], case["q_len"], case["heads"] // H
    lens = s["lens"].tolist()
    if 4 * case["heads"] * T * D * sum(_span(case, n) for n in lens) > 4e12:   # fp64 on this card: over 20 s
        return None
    o = torch.zeros(B, T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    window = case["window"]
    for b, n in enumerate(lens):
        first = _first(case, n)
        pos = torch.cat((torch.arange(min(case["sinks"], first)), torch.arange(first, n))).cuda()
        if "table" in s:
            page, slot = s["table"][b].long().index_select(0, pos // P), pos % P
        else:
            page, slot = torch.full_like(pos, b), pos
        own_pos = [n - T + i for i in range(T)]
        hide = torch.full((T, 1, len(pos)), -math.inf, dtype=torch.float64, device="cuda")
        for i, p in enumerate(own_pos):
            see = pos <= p
            if window:
                see = see & ((pos < case["sinks"]) | (pos > p - window))
            hide[i, 0, see] = 0.0
        for h in range(H):
            if op == "decode4":
                size = s["k"][0].shape[2]
                at = (page * H + h) * size + slot
                k, v = _exact_values4(s["k"], s["k_scale"], at), _exact_values4(s["v"], s["v_scale"], at)
            else:
                size = s["k"].shape[1]
                at = (page * size + slot) * H + h
                k, v = (x.view(-1, D).view(torch.uint8 if x.element_size() == 1 else x.dtype).index_select(0, at)
                        .view(x.dtype).double() * float(np.float32(t)) for x, t in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,nd->tgn", q, k) * s["scale"] + hide
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[b, :, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, v)
            lse[b, :, h * G:(h + 1) * G] = z
    return o, lse
