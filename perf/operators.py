"""Workloads of the speculative-decoding operators over a KV cache, with their plain forms.

Four operators, as one step of speculative decoding calls them:

  tables   block tables and slot maps built on the GPU from request lengths
  write    new K/V rows written to the cache's slots, quantised for an FP8 cache
  tree     attention of a tree of drafted tokens over the cache
  compact  the accepted path's K/V rows moved to the front of the drafted tail

``run`` computes each in its plain form (elementary torch operations in fp32)
or, where ``own`` is set, with the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 running requests, one new token each: nothing but latency
        dict(name="tables_step", op="tables", batch=64, page=16, old_min=1, old_max=16384, new_min=1, new_max=1,
             held_extra=0),
        # a prefill wave: ragged prompts of up to 8192 tokens, some pages still held from rejected drafts
        dict(name="tables_prefill", op="tables", batch=384, page=16, old_min=0, old_max=512, new_min=1,
             new_max=8192, held_extra=2),
        # the K/V rows of one decoding step of 64 requests with 8 drafted tokens each
        dict(name="write_step", op="write", tokens=512, slots=65536, kv_heads=8, dim=128, dtype="bf16", kv="same",
             pad=0, strided=True),
        # a prefill's rows, cut out of a fused QKV projection, into a 16-bit cache
        dict(name="write_prefill", op="write", tokens=32768, slots=65536, kv_heads=8, dim=128, dtype="bf16",
             kv="same", pad=1000, strided=True),
        # a prefill's rows quantised into an FP8 cache
        dict(name="write_prefill_e4m3", op="write", tokens=65536, slots=131072, kv_heads=8, dim=128, dtype="bf16",
             kv="e4m3", pad=77, strided=True),
        # after verification: up to 8 accepted of 64 drafted tokens, 64 requests, paged GQA cache
        dict(name="compact_step", op="compact", batch=64, tree=64, accept=8, kv_heads=8, dim=128, page=16,
             len_min=64, len_max=512, kv="bf16"),
        # the same with many requests and all 32 heads in the cache, paths of up to 32 tokens
        dict(name="compact_large", op="compact", batch=320, tree=64, accept=32, kv_heads=32, dim=128, page=64,
             len_min=64, len_max=128, kv="bf16"),
        # one short request of a small MHA model, 8 drafted tokens: latency
        dict(name="tree_short", op="tree", batch=1, heads=32, kv_heads=32, dim=128, tree=8, ragged=False, page=0,
             len_min=2048, len_max=2048, dtype="bf16", kv="same", shared=True),
        # ragged GQA-4 requests in a contiguous fp16 cache, trees of up to 32 nodes
        dict(name="tree_ragged", op="tree", batch=16, heads=32, kv_heads=8, dim=128, tree=32, ragged=True, page=0,
             len_min=512, len_max=8192, dtype="f16", kv="same", shared=False),
        # a ragged serving batch over 16-token pages, 16 nodes
        dict(name="tree_paged", op="tree", batch=64, heads=32, kv_heads=8, dim=128, tree=16, ragged=True, page=16,
             len_min=64, len_max=16384, dtype="bf16", kv="same", shared=False),
        # GQA-8 with full trees of 64 nodes (512 query rows a kv head): tensor-core bound
        dict(name="tree_wide", op="tree", batch=4, heads=64, kv_heads=8, dim=128, tree=64, ragged=False, page=64,
             len_min=32768, len_max=32768, dtype="bf16", kv="same", shared=True),
        # GQA-8 over an FP8 cache, 16 nodes
        dict(name="tree_e4m3", op="tree", batch=16, heads=64, kv_heads=8, dim=128, tree=16, ragged=False, page=64,
             len_min=4096, len_max=32768, dtype="bf16", kv="e4m3", shared=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["tables", "write", "compact", "tree", "tree", "tree"])
    if op == "tables":
        old = _log_int(rng, 1, 16384)
        new = _log_int(rng, 1, 8192)
        return dict(op=op, batch=_log_int(rng, 1, 1024), page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                    old_min=rng.randint(0, old), old_max=old, new_min=rng.randint(0, new), new_max=new,
                    held_extra=rng.choice([0, 0, 1, 3]))
    if op == "write":
        tokens = _log_int(rng, 1, 65536)
        return dict(op=op, tokens=tokens, slots=tokens + _log_int(rng, 1, 65536), kv_heads=rng.choice([1, 2, 5, 8, 32]),
                    dim=rng.choice([64, 128, 256]), dtype=rng.choice(["bf16", "f16"]),
                    kv=rng.choice(["same", "e4m3", "e5m2"]), pad=rng.randint(0, 300), strided=rng.random() < 0.5)
    if op == "compact":
        tree = _log_int(rng, 2, 128)
        return dict(op=op, batch=_log_int(rng, 1, 256), tree=tree, accept=rng.randint(1, min(tree, 32)),
                    kv_heads=rng.choice([1, 2, 8, 32]), dim=rng.choice([64, 128, 256]),
                    page=rng.choice([0, 1, 16, 64]), len_min=tree, len_max=tree + _log_int(rng, 1, 512),
                    kv=rng.choice(["bf16", "f16", "e4m3"]))
    kv_heads, group = rng.choice([(32, 1), (8, 1), (8, 4), (8, 8), (4, 3), (1, 16), (2, 7)])
    tree = _log_int(rng, 1, 128)
    lo = _log_int(rng, 1, 8192)
    return dict(op="tree", batch=_log_int(rng, 1, 48), heads=kv_heads * group, kv_heads=kv_heads,
                dim=rng.choice([64, 128, 128, 256]), tree=tree, ragged=rng.random() < 0.5,
                page=rng.choice([0, 0, 4, 16, 32, 64, 128]), len_min=lo, len_max=lo + _log_int(rng, 1, 16384),
                dtype=rng.choice(["bf16", "f16"]), kv=rng.choice(["same", "same", "e4m3", "e5m2"]),
                shared=rng.random() < 0.3)


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
        # the plain form's fp32 copies of the whole cache and the scores stay within the card
        if c["op"] == "tree" and c["batch"] * c["len_max"] * (c["kv_heads"] * c["dim"] * 8 + c["heads"] * c["tree"] * 16) > 60e9:
            continue
        return c


# ---------------------------------------------------------------- inputs

def _grid(lo, hi, n):
    """n whole numbers spread evenly from lo to hi (one: hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tree_grid(case):
    if not case["ragged"]:
        return [case["tree"]] * case["batch"]
    return _grid(max(1, case["tree"] // 2), case["tree"], case["batch"])


def _parents(rng, n):
    """Parents of a drafted tree's nodes in order: a node hangs under an earlier one or under the context."""
    return [rng.randint(max(-1, i - 1 - n // 4), i - 1) for i in range(n)]


def _mask_words(parents, words):
    """Visibility bits: a node sees itself and its ancestors."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return [[(b >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for b in bits]


def _rows(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype) if \
        math.prod(shape) < (1 << 26) else torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).to(dtype)


def _cache(gen, rows, kv_heads, dim, kv):
    return _rows(gen, (rows, kv_heads, dim), _T[kv])


def _paged(rng, gen, lens, page, spare):
    """(block table, pages): requests' pages scattered over a pool with spare pages; unused entries are -1."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(need))
    n = torch.tensor(need, device="cuda")
    first = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j[None, :]).clamp_(max=pages - 1)
    table = torch.where(j[None, :] < n[:, None], order[at], torch.full_like(order[at], -1))
    return table.contiguous(), pages


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op == "tables":
        B, page = case["batch"], case["page"]
        old, new = _grid(case["old_min"], case["old_max"], B), _grid(case["new_min"], case["new_max"], B)
        rng.shuffle(old)
        rng.shuffle(new)
        held = [-(-o // page) + rng.randint(0, case["held_extra"]) for o in old]
        width = -(-(case["old_max"] + case["new_max"]) // page) + case["held_extra"]
        used = sum(max(0, -(-(o + n) // page) - h) for o, n, h in zip(old, new, held))
        table, pages = _paged(rng, gen, [h * page for h in held], page, used + 64)
        full = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        w = min(width, table.shape[1])
        full[:, :w] = table[:, :w]
        taken = torch.zeros(pages, dtype=torch.bool, device="cuda")
        taken[table[table >= 0].long()] = True
        free = torch.nonzero(~taken).flatten()
        free = free[torch.randperm(free.numel(), generator=gen, device="cuda")].to(torch.int32)
        s.update(old=_i32(old), new=_i32(new), held=_i32(held), table=full, free=free,
                 free_count=_i32([free.numel()]), pages=pages, max_tokens=sum(new) + (-sum(new)) % 64)
    elif op == "write":
        n, H, D = case["tokens"], case["kv_heads"], case["dim"]
        dt = _T[case["dtype"]]
        if case["strided"]:   # K and V as the last columns of a fused GQA-4 projection's output
            qkv = _rows(gen, (n, 6 * H * D), dt, 1.5)
            s["k_new"], s["v_new"] = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (4, 5))
        else:
            s["k_new"], s["v_new"] = (_rows(gen, (n, H, D), dt, 1.5) for _ in range(2))
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int64)
        if case["pad"]:   # the padded end of a captured batch
            slots[max(1, n - case["pad"]):] = -1
        kv = case["dtype"] if case["kv"] == "same" else case["kv"]
        s.update(slots=slots, k=_cache(gen, case["slots"], H, D, kv), v=_cache(gen, case["slots"], H, D, kv),
                 k_scale=0.02 * (1 + rng.random()) if case["kv"] != "same" else 1.0,
                 v_scale=0.02 * (1 + rng.random()) if case["kv"] != "same" else 1.0)
    elif op == "compact":
        B, T, page = case["batch"], case["tree"], case["page"]
        lens = _grid(case["len_min"], case["len_max"], B)
        rng.shuffle(lens)
        n = _grid(1, case["accept"], B)
        rng.shuffle(n)
        paths = [sorted(rng.sample(range(T), k)) + [-1] * (case["accept"] - k) for k in n]
        if page:
            s["table"], s["pages"] = _paged(rng, gen, lens, page, 8)
            rows = (s["pages"], page)
        else:
            rows = (B, case["len_max"])
        s.update(lens=_i32(lens), accepted=_i32(paths), accept_lens=_i32(n),
                 k=_cache(gen, math.prod(rows), case["kv_heads"], case["dim"], case["kv"]).view(*rows, case["kv_heads"], case["dim"]),
                 v=_cache(gen, math.prod(rows), case["kv_heads"], case["dim"], case["kv"]).view(*rows, case["kv_heads"], case["dim"]))
    else:
        B, T, page, H, D = case["batch"], case["tree"], case["page"], case["kv_heads"], case["dim"]
        lens, trees = _grid(case["len_min"], case["len_max"], B), _tree_grid(case)
        rng.shuffle(lens)
        words = -(-T // 64)
        masks = [_mask_words(_parents(rng, T), words) for _ in range(1 if case["shared"] else B)]
        masks = torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).cuda()
        kv = case["dtype"] if case["kv"] == "same" else case["kv"]
        if page:
            s["table"], pages = _paged(rng, gen, lens, page, 8)
            rows = (pages, page)
        else:
            rows = (B, case["len_max"])
        s.update(q=_rows(gen, (B, T, case["heads"], D), _T[case["dtype"]], 2.0),
                 k=_cache(gen, math.prod(rows), H, D, kv).view(*rows, H, D),
                 v=_cache(gen, math.prod(rows), H, D, kv).view(*rows, H, D),
                 mask=masks[0].contiguous() if case["shared"] else masks, lens=_i32(lens),
                 trees=_i32(trees) if case["ragged"] else None, scale=1.0 / math.sqrt(D),
                 k_scale=0.5 if case["kv"] != "same" else 1.0, v_scale=1.5 if case["kv"] != "same" else 1.0)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_tables(s):
    c = s["case"]
    B, P, N = c["batch"], c["page"], s["max_tokens"]
    old, new, held = s["old"].long(), s["new"].long(), s["held"].long()
    need = ((old + new + P - 1) // P - held).clamp_(min=0)
    first = torch.cumsum(need, 0) - need                     # ordinal of a request's first new page
    cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    table, free = s["table"], s["free"]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    ordinal = first[:, None] + col - held[:, None]
    taken = free[(s["free_count"].long() - 1 - ordinal).clamp_(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, taken, table))
    i = torch.arange(N, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True).clamp_(max=B - 1)
    pos = old[b] + i - cu[b]
    page = table[b, (pos // P).clamp_(max=table.shape[1] - 1)].long()
    slots = torch.where(i < cu[B], page * P + pos % P, torch.full_like(i, -1))
    return (table, slots, cu.to(torch.int32), (old + new).to(torch.int32), (held + need).to(torch.int32),
            (s["free_count"] - need.sum()).to(torch.int32))


def _plain_write(s):
    slots = s["slots"]
    ok = slots >= 0
    at = slots[ok]
    for new, cache, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        rows = new[ok]
        if cache.element_size() == 1:
            top = torch.finfo(cache.dtype).max
            rows = (rows.float() / torch.tensor(scale, dtype=torch.float32, device="cuda")).clamp(-top, top).to(cache.dtype)
            cache.view(torch.uint8)[at] = rows.view(torch.uint8)
        else:
            cache[at] = rows
    return s["k"], s["v"]


def _rows_of(s, pos):
    """Flat cache rows of positions pos [B, n] of every request."""
    B = pos.shape[0]
    if "table" in s:
        P = s["k"].shape[1]
        page = torch.gather(s["table"], 1, (pos // P).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
        return page * P + pos % P
    return torch.arange(B, device="cuda")[:, None] * s["k"].shape[1] + pos


def _plain_compact(s):
    c = s["case"]
    base = s["lens"].long() - c["tree"]
    j = torch.arange(c["accept"], device="cuda")[None, :]
    ok = j < s["accept_lens"][:, None]
    src = _rows_of(s, base[:, None] + s["accepted"].long().clamp(min=0))[ok]
    dst = _rows_of(s, base[:, None] + j.expand(c["batch"], -1))[ok]
    for t in (s["k"], s["v"]):
        flat = t.view(-1, c["kv_heads"], c["dim"])
        if t.element_size() == 1:
            flat = flat.view(torch.uint8)
        flat[dst] = flat[src]
    return s["k"], s["v"], (base + s["accept_lens"]).to(torch.int32)


def _plain_tree(s):
    c = s["case"]
    B, T, H, D = c["batch"], c["tree"], c["kv_heads"], c["dim"]
    G, L = c["heads"] // H, c["len_max"]
    pos = torch.arange(L, device="cuda")[None, :].expand(B, L)
    flat = _rows_of(s, pos)

    def rows(t):   # [B, H, L, D] fp32
        t = t.view(-1, H, D)
        if t.element_size() == 1:
            return t.view(torch.uint8)[flat].view(t.dtype).float().transpose(1, 2)
        return t[flat].float().transpose(1, 2)

    lens = s["lens"].long()
    trees = s["trees"].long() if s["trees"] is not None else torch.full_like(lens, T)
    node = pos - (lens - trees)[:, None]                     # tree node at a position; negative: context
    bits = ((s["mask"][..., None] >> torch.arange(64, device="cuda")) & 1).flatten(-2).bool()   # [(B,) T, 64 W]
    bits = bits.expand(B, T, bits.shape[-1])
    sees = torch.gather(bits, 2, node.clamp(0, T - 1)[:, None, :].expand(B, T, L))
    i = torch.arange(T, device="cuda")[None, :, None]
    sees = (sees | (node < 0)[:, None, :]) & (pos < lens[:, None])[:, None, :] & (i < trees[:, None, None])
    sees = sees & (lens[:, None, None] - trees[:, None, None] + i >= 0)
    sees = sees[:, None, :, None, :]                         # [B, 1, T, 1, L]
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    x = torch.matmul(q, rows(s["k"]).transpose(2, 3)).mul_(s["scale"] * s["k_scale"]).view(B, H, T, G, L)
    x = x.masked_fill_(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = x.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, T * G, L), rows(s["v"])).view(B, H, T, G, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-38) * s["v_scale"], torch.zeros_like(o))
    lse = (m0 + total.log()).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D), lse.permute(0, 2, 1, 3).reshape(B, T, H * G))


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    if own:
        import decode_attention_decoding_gb300 as fd
        if c["op"] == "tables":
            return fd.fd_build_tables(s["old"], s["new"], s["table"], s["free"], s["free_count"], c["page"],
                                      s["pages"], s["max_tokens"], held_pages=s["held"])
        if c["op"] == "write":
            fd.fd_cache_write(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"])
            return s["k"], s["v"]
        if c["op"] == "compact":
            lens = fd.fd_cache_compact(s["k"], s["v"], s["lens"], s["accepted"], s["accept_lens"], c["tree"],
                                       block_table=s.get("table"))
            return s["k"], s["v"], lens
        if "workspace" not in s:   # a program keeps one workspace for its calls
            s["workspace"] = fd.make_tree_workspace(c["batch"], c["tree"], c["heads"], c["kv_heads"], c["dim"])
        more = dict(tree_lens=s["trees"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                    workspace=s["workspace"])
        if c["page"]:
            return fd.fd_tree_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["mask"], **more)
        return fd.fd_tree_decode(s["q"], s["k"], s["v"], s["lens"], s["mask"], **more)
    return {"tables": _plain_tables, "write": _plain_write, "compact": _plain_compact, "tree": _plain_tree}[c["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "tables":
        B, P = case["batch"], case["page"]
        old, new = _grid(case["old_min"], case["old_max"], B), _grid(case["new_min"], case["new_max"], B)
        tokens = sum(new)
        pages = sum(-(-n // P) for n in new)
        # lengths and held pages in and out, the free pages read and entered, a slot a token
        return {"bytes": 24 * B + 8 * pages + 8 * (tokens + (-tokens) % 64), "flops": 2 * tokens}
    if op == "write":
        row = case["kv_heads"] * case["dim"]
        n = max(min(case["tokens"], 1), case["tokens"] - case["pad"])
        out = 2 if case["kv"] == "same" else 1
        return {"bytes": 2 * n * row * (2 + out) + 8 * case["tokens"], "flops": 0 if out == 2 else 2 * n * row}
    if op == "compact":
        n = sum(_grid(1, case["accept"], case["batch"]))
        row = case["kv_heads"] * case["dim"] * (1 if case["kv"] in _FP8_MAX else 2)
        return {"bytes": 2 * 2 * n * row + 4 * n + 16 * case["batch"], "flops": 0}
    B, T, H, D = case["batch"], case["tree"], case["kv_heads"], case["dim"]
    G = case["heads"] // H
    lens, trees = _grid(case["len_min"], case["len_max"], B), _tree_grid(case)
    # K and V once, q and o once
    eb = 2 if case["kv"] == "same" else 1
    kv = 2 * eb * H * D * sum(lens)
    return {"bytes": kv + 6 * B * T * H * G * D + 4 * B * T * H * G,
            "flops": 4 * H * G * D * sum(n * t for n, t in zip(sorted(lens), trees))}


# ---------------------------------------------------------------- the definition in 64 bits

def _fp8_exact(x, kv):
    """x (fp64) rounded to the nearest FP8 value, ties to even, saturating."""
    mant, low = (3, -6) if kv == "e4m3" else (2, -14)
    _, e = torch.frexp(x)                       # |x| in [2^(e-1), 2^e)
    step = torch.exp2((torch.clamp(e - 1, min=low) - mant).double())
    top = _FP8_MAX[kv]
    return torch.clamp(torch.round(x / step) * step, -top, top)   # torch.round: half to even


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        B, P = case["batch"], case["page"]
        old, new, held, free = (s[k].tolist() for k in ("old", "new", "held", "free"))
        table, left = s["table"].cpu().numpy().copy(), s["free_count"].item()
        slots, cu, held_out = [], [0], []
        for b in range(B):
            have = held[b]
            while have * P < old[b] + new[b]:
                left -= 1
                table[b, have] = free[left]
                have += 1
            held_out.append(have)
            pos = np.arange(old[b], old[b] + new[b], dtype=np.int64)
            slots.append(table[b][pos // P].astype(np.int64) * P + pos % P)
            cu.append(cu[-1] + new[b])
        slots.append(np.full(s["max_tokens"] - cu[-1], -1, dtype=np.int64))
        i32 = lambda v: np.array(v, dtype=np.int32)  # noqa: E731
        return (table, np.concatenate(slots), i32(cu), i32([o + n for o, n in zip(old, new)]), i32(held_out), i32([left]))
    if op == "write":
        out = []
        for x, cache, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
            x, y = x.double(), cache.double()
            if case["kv"] != "same":   # the scale is the fp32 number that a call takes
                x = _fp8_exact(x / float(np.float32(scale)), case["kv"])
            live = torch.nonzero(s["slots"] >= 0).flatten()
            y.index_copy_(0, s["slots"].index_select(0, live), x.index_select(0, live))
            out.append(y)
        return tuple(out)
    if op == "compact":
        lens, acc, n = s["lens"].tolist(), s["accepted"].tolist(), s["accept_lens"].tolist()
        table = s["table"].tolist() if "table" in s else None
        P = s["k"].shape[1]
        row = (lambda b, t: table[b][t // P] * P + t % P) if table else (lambda b, t: b * P + t)  # noqa: E731
        src = [row(b, lens[b] - case["tree"] + acc[b][j]) for b in range(len(lens)) for j in range(n[b])]
        dst = [row(b, lens[b] - case["tree"] + j) for b in range(len(lens)) for j in range(n[b])]
        src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
        out = []
        for t in (s["k"], s["v"]):
            y = t.double().view(-1, case["kv_heads"], case["dim"])
            out.append(y.index_copy(0, dst, y.index_select(0, src)).view(t.shape))
        return (*out, np.array([a - case["tree"] + m for a, m in zip(lens, n)], dtype=np.int32))
    B, T, H, D = case["batch"], case["tree"], case["kv_heads"], case["dim"]
    G = case["heads"] // H
    lens = s["lens"].tolist()
    if 4 * case["heads"] * T * D * sum(lens) > 4e12:   # fp64 on this card: over 20 s
        return None
    trees = s["trees"].tolist() if s["trees"] is not None else [T] * B
    words = s["mask"].cpu().numpy().view(np.uint64)
    o = torch.zeros(B, T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, t = lens[b], trees[b]
        first = max(0, t - n)                   # nodes before the cache's first position do not exist
        if n == 0 or first >= t:
            continue
        if "table" in s:
            page = s["table"][b].long().clamp(min=0).repeat_interleave(case["page"])[:n]
            at = page * case["page"] + torch.arange(n, device="cuda") % case["page"]
            k, v = (x.view(-1, H, D).view(torch.uint8 if x.element_size() == 1 else x.dtype).index_select(0, at).view(x.dtype).double()
                    for x in (s["k"], s["v"]))
        else:
            k, v = s["k"][b, :n].double(), s["v"][b, :n].double()
        w = words if case["shared"] else words[b]
        see = np.zeros((t - first, n), dtype=bool)
        see[:, :max(0, n - t)] = True
        for i in range(first, t):
            for j in range(first, t):
                see[i - first, n - t + j] = bool((int(w[i][j // 64]) >> (j % 64)) & 1)
        hide = torch.where(torch.from_numpy(see).cuda(), 0.0, -math.inf).double()
        for h in range(H):
            q = s["q"][b, first:t, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,nd->tgn", q, k[:, h]) * (s["scale"] * s["k_scale"]) + hide[:, None, :]
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[b, first:t, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, v[:, h]) * s["v_scale"]
            lse[b, first:t, h * G:(h + 1) * G] = z
    return o, lse
