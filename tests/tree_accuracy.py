"""How near a tree attention has to come to the 64-bit form by norm, and a model
of its arithmetic with parts that can be left out.

A bound for each element has to hold for the worst signs of n roundings, so for
thousands of positions it is far above what a right kernel does.  By norm, on V
of random signs, roundings add up as the outputs themselves do:
    ||O - ref|| <= 2^-16 ||ref||       over the rows and dims of a request.
  - a weight in two bf16 parts is off by at most 2^-8 2^-8 of itself: errors of
    independent signs, 2^-16 of ||ref|| if each were as large as it can be, and
    some 0.2 of that as they fall (uniform in either rounding);
  - an accumulator loses 1.7e-8 of itself at an MMA (measured on GB300), 256 of
    them between flushes: at most 4.4e-6 = 0.29 2^-16;
  - scores of a few units are off by less than 2^-20 (D / 16 fp32 steps), the
    exponential by 2^-22: 0.1 2^-16.
Weights of one 16-bit part alone are off by up to 2^-8 (bf16) or 2^-11 (fp16), and
by some 0.4 of that as they fall: 100 or 13 times the bound.  An accumulator of
40000 positions that is never flushed loses some 4e-5, nearly three times the
bound."""
import numpy as np
import torch

NORM_BOUND = 2.0 ** -16


def attention64(c, scale, ks=1.0, vs=1.0, device="cpu"):
    """O and LSE of a case in 64 bits, [B, T, Hq, D] and [B, T, Hq] (every row must see something)."""
    q, vis = (torch.from_numpy(c[n]).to(device) for n in ("q64", "vis"))
    B, T, hq, D = q.shape
    o, lse = torch.empty(B, T, hq, D, dtype=torch.float64), torch.empty(B, T, hq, dtype=torch.float64)
    for b in range(B):
        k, v = (torch.from_numpy(c[n][b]).to(device) for n in ("k64", "v64"))
        L, t, G = c["lens"][b], c["trees"][b], hq // k.shape[1]
        for g in range(k.shape[1]):
            s = torch.einsum("thd,nd->thn", q[b, :, g * G:(g + 1) * G], k[:, g]) * (scale * ks)
            s[:, :, L - t:].masked_fill_(~vis[b, :, None, :t], -torch.inf)
            top = torch.logsumexp(s, -1)
            o[b, :, g * G:(g + 1) * G] = (torch.exp(s - top[..., None]) @ v[:, g] * vs).cpu()
            lse[b, :, g * G:(g + 1) * G] = top.cpu()
    return o, lse


def norm_errors(o, ref):
    """||O - ref|| / ||ref|| of every request."""
    return [float((o[b].double().cpu() - ref[b]).norm() / ref[b].norm()) for b in range(len(ref))]


def cut(x, bits=25):
    """x to so many significant bits, towards zero; 25 lose 2e-8 a step on average, about what was measured."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, bits)), e - bits)


def model(q, k, v, scale, dtype, parts=2, flush=2048):
    """The kernel's arithmetic for rows q [n, D] over k, v [L, D]: weights in `parts` 16-bit parts,
    accumulators cut at every MMA of 16 positions and flushed into fp32 every `flush` positions."""
    t, shift = (torch.bfloat16, 1.0) if dtype == "bf16" else (torch.float16, 256.0)
    s = q @ k.T * scale
    p = torch.from_numpy(np.exp(s - s.max(-1, keepdims=True)) * shift).float()
    pieces, rest = [], p
    for _ in range(parts):
        piece = rest.to(t).float()
        pieces.append(piece.double().numpy())
        rest = rest - piece
    sums, acc = np.zeros((len(q), v.shape[1]), dtype=np.float32), np.zeros((len(q), v.shape[1]))
    for n in range(0, len(k), 16):
        for piece in pieces:
            acc = cut(acc + piece[:, n:n + 16] @ v[n:n + 16])
        if (n + 16) % flush == 0:
            sums, acc = sums + acc.astype(np.float32), np.zeros_like(acc)
    return (sums + acc.astype(np.float32)) / p.double().numpy().sum(-1, keepdims=True)
