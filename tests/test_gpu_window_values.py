"""Window and 4-bit attention on values at the ends of their types' ranges: large finite V behind weights that fp32 does
not hold, and infinities beside them."""
import math

import numpy as np
import pytest
import torch

import longcontext_util as u

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "e4m3", "e5m2", "e2m1"]
# query heads (of 2 kv heads) and new tokens: 1 (both parts of a weight in one MMA in fp16), 6 and 16 columns
COLUMNS = [(2, 1), (4, 3), (32, 1)]
# one tile or two; many tiles a warp and the joining of a CTA's warps; the joining of CTAs
SPLITS = [(40, 0), (3000, 1), (20000, 0)]


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def fill(c, i, x):
    """The case's K (i = 0) or V (1), in the tensors and in 64 bits, from values [L, hkv, D] that are rounded to its type."""
    name = ("k64", "v64")[i]
    if c["kv"] == "e2m1":
        codes, s = u.quantise4(torch.from_numpy(x).bfloat16(), 1.0)
        for j, y in enumerate((codes, s)):
            c["pool"][2 * i + j][0] = torch.from_numpy(y).transpose(0, 1)
        c[name][0] = u.values4(codes, s)
    else:
        t = torch.from_numpy(x).to(c["pool"][i].dtype)
        c["pool"][i][0] = t
        c[name][0] = t.double().numpy()


def case(kv, hq, T, L, q, seed):
    c = u.make_case(seed, 1, T, hq, 2, 128, [L], kv=kv)
    c["q"] = torch.full_like(c["q"], q)
    c["q64"] = c["q"].double().numpy()
    return c


def mean_bound(c, top):
    """Of the mean of the V rows `top` [L] that a token sees, taken with equal weights that are powers of 2 (exact in 16
    bits): each of n additions 2^-23 of what is added, O's division, its product and the joining of partials a few more."""
    L, T, G = c["lens"][0], c["q"].shape[1], c["q"].shape[2] // 2
    err = np.zeros(c["q"].shape)
    for i in range(T):
        at = u.sees(L, T, i, 0, 0) & top
        err[0, i] = ((at.sum() + 16) * 2.0 ** -22 * np.abs(c["v64"][0][at]).mean(0)).repeat(G, 0)
    return err


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("hq,T", COLUMNS)
@pytest.mark.parametrize("L,ctas", SPLITS)
@pytest.mark.parametrize("near", ["first", "last", "spread"])
@pytest.mark.parametrize("bad", [False, True])
def test_large_finite_values_vanish_and_infinities_stay(fd, kv, hq, T, L, ctas, near, bad):
    """Far rows score 256 nats and more below the near ones, weights of 2^-369, and hold numbers near their type's largest
    (bf16: 2^112, which 20000 rows of do not pass fp32's range): 0 in fp32, whichever tile, warp or CTA meets them first.
    An infinity among them stays one."""
    if bad and kv in ("e4m3", "e2m1"):
        pytest.skip("the type has no infinity")
    c = case(kv, hq, T, L, 4.0, 71)
    top = np.zeros(L, dtype=bool)
    if near == "spread":
        top[7::max(L // 5, 1)] = True
    else:
        at = {"first": 0, "last": L - 3 - T}[near]
        top[at:at + 3] = True
    k, v = np.zeros((L, 2, 128)), np.random.default_rng(5).standard_normal((L, 2, 128))
    k[~top] = -1.0
    v[~top] = {"bf16": 2.0 ** 112, "f16": 65504.0, "e4m3": 448.0, "e5m2": 57344.0, "e2m1": 2688.0}[kv]
    v[~top, :, 1::2] *= -1
    v[top, :, 96:] = 0.0
    if bad:
        far = np.nonzero(~top)[0]
        far = far[far < L - T]
        v[far[1], :, 5] = v[far[-2], :, 100] = math.inf
        v[far[-1], :, 6] = -math.inf
        v[far[0], :, 20], v[far[-1], :, 20] = math.inf, -math.inf
    fill(c, 0, k)
    fill(c, 1, v)
    o, lse = u.run(fd, c, 0.5, num_ctas=ctas, k_scale=1.0, v_scale=1.0)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    ref, ref_lse, _, _ = u.attention(c["q64"], c["k64"], c["v64"], c["lens"], 0, 0, 0.5)
    assert np.abs(lse - ref_lse).max() <= 2.0 ** -20        # ln of 3 to 6
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    inf = np.isinf(ref)
    assert bool(inf.any()) == bad and np.array_equal(o[inf], ref[inf])
    fin = np.isfinite(ref)
    off = np.abs(o[fin] - ref[fin])
    assert (off <= mean_bound(c, top)[fin] + 2.0 ** -149).all(), off.max()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("hq,T", COLUMNS)
@pytest.mark.parametrize("L,ctas", [(40, 0), (1500, 1), (6000, 0)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(fd, kv, hq, T, L, ctas, sign):
    """Scores of 0.7 2^e (or its negative), 0 and a little above that, each the same in many rows: the rows of the highest
    have equal weights, the others none from e = 8 on.  Of a product that fp32 rounds by more than 1, each weight has to
    mean the same."""
    rng = np.random.default_rng(L)
    level = rng.integers(0, 4, L)
    level[0] = level[L - T] = 3
    c = case(kv, hq, T, L, 3.0, 72)
    fill(c, 0, sign * np.array([-1.5, 0.0, 0.5, 1.5])[level][:, None, None] * np.ones((1, 2, 128)))
    fill(c, 1, rng.standard_normal((L, 2, 128)))
    top = c["k64"][0][:, 0, 0] * sign == (c["k64"][0][:, 0, 0] * sign).max()
    assert (top == (level == 3)).all()
    bound = mean_bound(c, top)
    for e in (8, 22, 23, 25, 26, 28, 33, 100):
        scale = sign * float(np.float32(0.7 * 2.0 ** e / 576))
        o, lse = u.run(fd, c, scale, num_ctas=ctas, k_scale=1.0, v_scale=1.0)
        ref, ref_lse, _, _ = u.attention(c["q64"], c["k64"], c["v64"], c["lens"], 0, 0, scale)
        # 576 dims' products are exact; the scale in log2 units, the product, the reference and ln 2: 2^-24 each, twice over
        assert (np.abs(lse.double().cpu().numpy() - ref_lse) <= 2.0 ** -20 + np.abs(ref_lse) * 2.0 ** -21).all(), e
        assert (np.abs(o.double().cpu().numpy() - ref) <= bound).all(), e


def test_one_request_s_not_a_numbers_do_not_hold_up_the_others(fd):
    """Columns whose weights are NaN are NaN whatever V holds, so nothing is looked for in their rows; and infinities are
    looked for once, not for each new token.  Measured: 1.0 times a clean call and 10, before 10.5 and 147; the limits of 3
    and 40 lie between."""
    B, L = 64, 8192
    k, v = (torch.randn(B, L, 1, 128, device="cuda").bfloat16() for _ in range(2))
    ws = fd.make_window_workspace(B, 16, 1, 128)

    def time(q):
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
        times = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                fd.fd_window_decode(q, k, v, None, L, out=out, lse=lse, workspace=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times), out

    q = torch.randn(B, 16, 1, 128, device="cuda").bfloat16()
    one = torch.randn(B, 8, 128, device="cuda").bfloat16()
    clean, clean_one = time(q)[0], time(one)[0]
    one[5, :, 3] = math.nan
    t, o = time(one)
    assert bool(o[5].isnan().all()) and bool(o[:5].isfinite().all()) and bool(o[6:].isfinite().all())
    assert t <= 3 * clean_one
    v[:, ::1000, 0, 7] = math.inf
    t, o = time(q)
    assert bool((o[..., 7] == math.inf).all()) and bool(o[..., 8:].isfinite().all())
    assert t <= 40 * clean
