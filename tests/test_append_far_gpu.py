"""GPU test of the rotation at the last positions that a cache can have (2^31 - 64): the angle's reduction loses nothing."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rotation_at_the_last_positions():
    """q is (1, 0) in each pair, so that the rotated query is (cos a, sin a), rounded to bf16.

    The angle in fp32 half turns is off by pi 2^-25, sine and cosine by 2 ulp (2^-23): together under 2^-22.  A value as far
    as that from what lies between the neighbouring bf16 numbers' halves is right; with an angle off by 4e-7, as of an fp64
    product and an fp64 1 / (2 pi) alone, some of these 5 million values are not."""
    import fine_grained_top_b200 as sa
    T, d, max_pages = 40000, 128, (2 ** 31 - 1) // 64
    last = max_pages * 64
    half = d // 2
    g = torch.Generator().manual_seed(3)
    inv = (0.5 + 0.5 * torch.rand(half, generator=g)).float()
    p = np.arange(last - T, last, dtype=np.int64)   # positions
    pt = torch.zeros(1, max_pages, dtype=torch.int32, device="cuda")
    n_pages = T // 64 + 2
    pt[0, -n_pages:] = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    q = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., :half] = 1
    nv = torch.from_numpy((p + 1).astype(np.int32)).cuda()
    cache = torch.zeros(n_pages * 64, d, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    out, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    sa.sa_cache_append(q, d, out, kv, d, kv, d, None, 0, nv, pt, max_pages, n_pages, 64, 0, 1, T, 1, d, 0, inv.cuda(), d, 0,
                       cache, cache.clone(), None, 0, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    out = out.view(T, d)
    # the exact angle: position times a 24-bit number is below 2^55, its turns to 2^-35 in 64 bits of mantissa
    m, e = np.frexp(inv.numpy())
    product = p[:, None].astype(np.longdouble) * np.ldexp(m, 24).astype(np.longdouble)
    turns = product * np.longdouble("0.15915494309189533576888376337251436203") * np.ldexp(np.longdouble(1), e - 24)
    a = 2 * np.pi * (turns - np.rint(turns)).astype(np.float64)
    for got, want in ((out[:, :half], np.cos(a)), (out[:, half:], np.sin(a))):
        bits = got.contiguous().cpu().view(torch.int16).to(torch.int32)
        value = lambda b: (b << 16).view(torch.float32).double().numpy()  # noqa: E731
        v, w = value(bits), torch.from_numpy(want).numpy()
        # halfway to the bf16 numbers on either side (in magnitude; the bits of one sign are in order)
        lo, hi = (v + value(bits - 1)) / 2, (v + value(bits + 1)) / 2
        lo = np.where((bits.numpy() & 0x7FFF) == 0, -np.abs(hi), lo)
        beyond = np.maximum(np.abs(w) - np.abs(hi), np.abs(lo) - np.abs(w))
        assert beyond.max() <= 2.0 ** -22, "%d values off, by up to %.3g" % ((beyond > 2.0 ** -22).sum(), beyond.max())
