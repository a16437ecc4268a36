"""GPU tests of the caches' append on a stream of the caller's while others are busy."""

import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_queries_made_by_the_append_belong_to_its_stream(q8):
    """The append runs on a stream of its own while the current one is busy for some 100 ms: what it returns is the rotated
    queries, then and when the current stream has caught up."""
    from fine_grained_top_b200.pipeline import KVCache
    B, T, Hq, d, D_I = 2, 5, 8, 128, 64
    g = torch.Generator().manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, kI, nv = bf(B * T, Hq, d), bf(B * T, d), bf(B * T, d), bf(B * T, D_I), ref.rows_of([70, 9], [5, 4], T).cuda()
    cache = KVCache(B, d, D_I, S_max=128, q8=q8)
    want = cache.append(q, k, v, kI, nv, T=T, q_out=torch.zeros_like(q))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)   # clock ticks
    got = cache.append(q, k, v, kI, nv, T=T, stream=side)
    with torch.cuda.stream(side):
        early = got.clone()
    side.synchronize()
    assert not torch.cuda.current_stream().query()   # it really was busy all the while
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == 0 and want[:9].any() and not want[9].any()
    assert torch.equal(early, want) and torch.equal(got, want)
