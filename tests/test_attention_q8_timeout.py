"""A wait of the 8-bit attention's pipeline that runs out: one product of one row is never issued, the wait for it gives up
after 20 ms, and the kernel leaves in order."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p(256)   # a fake, aligned, never dereferenced pointer


@pytest.fixture(scope="module")
def sa():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_top_b200 as m
    return m


@pytest.mark.parametrize("kw", [dict(limit_us=0), dict(limit_us=1000001), dict(B=0), dict(B=1025), dict(Hq=17), dict(Hq=0),
                                dict(ctas=0), dict(ctas=17), dict(lost=-1), dict(S_max=63), dict(S_max=100),
                                dict(S_max=65600), dict(status=None), dict(q=None), dict(out=None), dict(n_valid=None),
                                dict(q=ctypes.c_void_p(264))])
def test_health_check_refusals(sa, kw):
    a = dict(q=P, k=P, v=P, ks=P, vs=P, S_max=640, n_valid=P, B=3, Hq=16, scale=0.1, out=P, ctas=1, lost=0, limit_us=1000,
             status=P, stream=None)
    a.update(kw)
    assert sa._lib.sa_selftest_attn_q8_timeout(*a.values()) == sa.SA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("ctas,tiles", [(1, 5), (2, 2), (1, 1)])
def test_a_product_that_never_comes(sa, ctas, tiles):
    """S or P V of each tile in turn: the time-out is reported, the other rows are right, and so is the next call."""
    n, B, Hq, d, scale = (640 if tiles > 1 else 128), 3, 16, 128, 0.09
    g = torch.Generator().manual_seed(tiles)
    codes = lambda: torch.randn(B * n, d, generator=g).mul(60).to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    kc, vc, s = codes(), codes(), torch.full((B * n // 64,), 2.0 ** -7, device="cuda")
    q = torch.randn(B, Hq, d, generator=g).bfloat16().cuda()
    nv = torch.tensor([n, n - 5, n - 70], dtype=torch.int32, device="cuda")

    def run(lost):
        out, status = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        sa.sa_selftest_attn_q8_timeout(q, kc, vc, s, s, n, nv, B, Hq, scale, out, ctas, lost, 20000, status)
        torch.cuda.synchronize()
        return out, int(status.item())

    def plain():
        out, status = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        sa.sa_sparse_attn_q8(q, kc, vc, s, s, 64, None, 0, 0, 64, n, nv, None, 0, n, B, 1, Hq, d, scale, out, None, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return out

    before = plain()
    whole, st = run(2 * tiles + 2)   # no such tile: an ordinary call
    # one row's two runs differ in the order of fp32 sums and an output rounding at most
    assert st == 0 and torch.allclose(whole.float(), before.float(), rtol=2.0 ** -7, atol=2.0 ** -12)
    for lost in range(2 * tiles):
        out, st = run(lost)
        assert st == sa.SA_DEV_TIMEOUT, lost
        assert torch.equal(out[1:], whole[1:]), lost
        assert torch.equal(plain(), before), lost
