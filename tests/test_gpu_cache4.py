"""fd_cache_write4 and fd_cache_read4 on the GPU, against their definitions."""
import numpy as np
import pytest
import torch

import longcontext_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def empty(fd, pages, h, page, d):
    """A cache that holds a pattern, on the CPU: codes and scales as uint8."""
    g = torch.Generator().manual_seed(pages)
    byte = lambda w: torch.randint(0, 256, (pages, h, page, w), generator=g, dtype=torch.uint8)  # noqa: E731
    return [byte(d // 2), byte(d // 16), byte(d // 2), byte(d // 16)]


def rows(n, h, d, dtype, seed, stride=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, stride or h * d, generator=g) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g).float())
    return x.to(dtype)[:, :h * d].unflatten(1, (h, d))


def expected(cache, slots, new, scales, page):
    out = [t.clone() for t in cache]
    for i, (x, t) in enumerate(zip(new, scales)):
        codes, s = u.quantise4(x, t)
        for j, slot in enumerate(slots):
            if 0 <= slot < cache[0].shape[0] * page:
                out[2 * i][slot // page, :, slot % page] = torch.from_numpy(codes[j])
                out[2 * i + 1][slot // page, :, slot % page] = torch.from_numpy(s[j])
    return out


def same(got, ref):
    for i, (a, b) in enumerate(zip(got, ref)):
        a = a.cpu().view(torch.uint8)
        if i % 2:   # any NaN is a NaN
            a, b = (torch.where((x & 127) == 127, torch.full_like(x, 127), x) for x in (a, b))
        assert torch.equal(a, b), f"tensor {i}: {int((a != b).sum())} of {a.numel()} bytes differ"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("h,page,pages,n", [(1, 1, 40, 17), (8, 16, 20, 300), (5, 24, 9, 200), (2, 7, 31, 1), (32, 64, 3, 150), (3, 500, 2, 777)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_write(fd, D, h, page, pages, n, dtype):
    """Every byte of the cache afterwards: the named slots', and all others as they were."""
    cache = empty(fd, pages, h, page, D)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[::5] = -1
    k, v = rows(n, h, D, dtype, 1, h * D + 40), rows(n, h, D, dtype, 2)
    n = len(slots)
    k, v = k[:n], v[:n]
    dev = fd.Cache4(*(t.cuda() for t in cache))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_dev = torch.empty(n, h * D + 40, dtype=dtype, device="cuda")[:, :h * D].unflatten(1, (h, D))
    k_dev.copy_(k)
    fd.fd_cache_write4(k_dev, v.cuda(), slots.cuda(), dev, k_scale=0.03, v_scale=1.7, device_status=status)
    same(dev, expected(cache, slots.tolist(), (k, v), (0.03, 1.7), page))
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t", [1.0, 2.0 ** -9, 0.037, 1e-30, 1e30])
def test_write_edge_values(fd, dtype, t):
    """Blocks of zeros and negative zeros, one element, ties of the codes and of the scale, subnormals, the largest
    numbers, infinities, NaN; tensor scales whose units leave the fast division's range."""
    top = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    blocks = [[0.0] * 16, [-0.0] * 16, [1.0] + [0.0] * 15, [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6],
              [6 * 1.0625] + [0.5] * 15, [6 * 1.1875] + [0.5] * 15, [tiny] * 16, [tiny / 4, -tiny / 2] * 8, [top, -top] * 8,
              [top, 1.0] * 8, [float("inf"), 1.0, -1.0, 0.0] * 4, [float("-inf")] * 16, [float("nan")] + [1.0] * 15, [1.0] * 15 + [float("nan")],
              [2688.0] * 16, [2880.0, -1344.0] * 8, [6 * 2.0 ** -9] * 16, [6 * 2.0 ** -10] * 16, [6 * 2.0 ** -10 * 1.01] * 16]
    blocks += [[x * s for x in blocks[3]] for s in (3.0, 0.4375, 104.0, t, 13 * t)]
    x = torch.tensor(blocks, dtype=torch.float64).to(dtype).reshape(len(blocks) // 4, 1, 64)
    n = x.shape[0]
    cache = empty(fd, n, 1, 1, 64)
    dev = fd.Cache4(*(y.cuda() for y in cache))
    slots = torch.arange(n)
    fd.fd_cache_write4(x.cuda(), x.cuda(), slots.cuda(), dev, k_scale=t, v_scale=t)
    same(dev, expected(cache, slots.tolist(), (x, x), (t, t), 1))


def test_write_every_number_against_every_scale(fd):
    """The fast division at every 16-bit mantissa and block scale: blocks whose largest element sets the scale, the
    others all mantissas between it and 0."""
    m = torch.arange(128) / 128 + 1
    tops = (torch.arange(8) / 8 + 1) * 6
    x = torch.cat([torch.stack([top.expand(128), *(m * 2.0 ** -e for e in range(-2, 4)), *(-m * 2.0 ** -e for e in range(-2, 4)), m / 32, m / 64, m * 0], 1)
                   for top in tops]).bfloat16()
    x = x.clamp(-6 * 1.9, 6 * 1.9).reshape(-1, 1, 64)
    n = x.shape[0]
    for t in (1.0, 0.0131, 0.7):
        cache = empty(fd, n, 1, 1, 64)
        dev = fd.Cache4(*(y.cuda() for y in cache))
        y = (x.float() * t).bfloat16()
        fd.fd_cache_write4(y.cuda(), y.cuda(), torch.arange(n).cuda(), dev, k_scale=t, v_scale=t)
        same(dev, expected(cache, list(range(n)), (y, y), (t, t), 1))


def test_bad_slots_are_reported(fd):
    cache = empty(fd, 4, 2, 16, 64)
    x = rows(5, 2, 64, torch.bfloat16, 3)
    slots = torch.tensor([3, 64, -5, 1 << 40, 63])
    dev = fd.Cache4(*(t.cuda() for t in cache))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd.fd_cache_write4(x.cuda(), x.cuda(), slots.cuda(), dev, device_status=status)
    same(dev, expected(cache, slots.tolist(), (x, x), (1.0, 1.0), 16))
    assert int(status) == fd.FD_DEVICE_STATUS_BAD_SLOT
    status.zero_()
    out = torch.full((5, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    fd.fd_cache_read4(slots.cuda(), dev, k_out=out, v_out=out.clone(), device_status=status)
    assert int(status) == fd.FD_DEVICE_STATUS_BAD_SLOT
    assert bool((out[1:4] == 7.0).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("h,page,pages,n", [(1, 1, 40, 17), (8, 16, 20, 300), (5, 24, 9, 200), (3, 500, 2, 777)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_read(fd, D, h, page, pages, n, dtype):
    """Every code under every scale (the cache holds random bytes), slots named twice, rows of negative slots left."""
    cache = empty(fd, pages, h, page, D)
    g = torch.Generator().manual_seed(n)
    slots = torch.randint(0, pages * page, (n,), generator=g)
    slots[::7] = -1
    wide = torch.full((n, h * D + 8), 5.0, dtype=dtype, device="cuda")
    k_out, v_out = wide[:, :h * D].unflatten(1, (h, D)), torch.full((n, h, D), 5.0, dtype=dtype, device="cuda")
    dev = fd.Cache4(*(t.cuda() for t in cache))
    k, v = fd.fd_cache_read4(slots.cuda(), dev, k_out=k_out, v_out=v_out, k_scale=0.3, v_scale=2.0)
    assert k.data_ptr() == k_out.data_ptr() and bool((wide[:, h * D:] == 5.0).all())
    for got, i, t in ((k, 0, 0.3), (v, 2, 2.0)):
        x = u.values4(cache[i].numpy(), cache[i + 1].numpy())
        x = x[slots.numpy() // page, :, slots.numpy() % page].astype(np.float32) * np.float32(t)   # code * s is exact
        x = torch.from_numpy(x).to(dtype)
        x[slots < 0] = 5.0
        assert torch.equal(torch.nan_to_num(got.cpu(), 1234.0), torch.nan_to_num(x, 1234.0))


def test_read_into_new_tensors(fd):
    cache = [t.cuda() for t in empty(fd, 3, 2, 16, 128)]
    k, v = fd.fd_cache_read4(torch.tensor([5, -1], device="cuda"), fd.Cache4(*cache))
    assert k.shape == v.shape == (2, 2, 128) and k.dtype is torch.bfloat16 and not bool(k[1].any())


def test_cache_beyond_4_gb(fd):
    """Slots whose codes lie past 2^32 bytes."""
    pages, h, page, D = 1100, 8, 4096, 256
    codes = torch.empty(pages, h, page, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, h, page, D // 16, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 32
    slots = torch.tensor([pages * page - 1, 0, 1024 * page + 5, 1023 * page + 4095, 600 * page], device="cuda")
    x, y = rows(5, h, D, torch.bfloat16, 9), rows(5, h, D, torch.bfloat16, 10)
    cache = fd.Cache4(codes, scales, codes.clone(), scales.clone())
    fd.fd_cache_write4(x.cuda(), y.cuda(), slots, cache)
    for got, ref in zip(fd.fd_cache_read4(slots, cache, torch.float16), (x, y)):
        assert torch.equal(got.cpu(), torch.from_numpy(u.values4(*u.quantise4(ref, 1.0))).to(torch.float16))


def test_python_checks(fd):
    cache = fd.make_cache4(4, 2, 16, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    fd.fd_cache_write4(x, x, slots - 1, cache)
    for bad in (lambda: fd.fd_cache_write4(x.float(), x.float(), slots, cache), lambda: fd.fd_cache_write4(x, x.half(), slots, cache),
                lambda: fd.fd_cache_write4(x, x, slots[:2], cache), lambda: fd.fd_cache_write4(x, x, slots.int(), cache),
                lambda: fd.fd_cache_write4(x[:, :1], x[:, :1], slots, cache),
                lambda: fd.fd_cache_write4(x, x, slots, cache._replace(v_codes=cache.k_codes[:3])),
                lambda: fd.fd_cache_write4(x, x, slots, cache._replace(v_scales=cache.v_scales.view(torch.int8))),
                lambda: fd.fd_cache_write4(x, x, slots, cache._replace(k_codes=cache.k_codes.transpose(1, 2)))):
        with pytest.raises(ValueError):
            bad()
