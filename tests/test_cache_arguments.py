"""Host checks of KVCache.append: rows of another width, or another number of them, are refused (no GPU: the checks run
before any CUDA call)."""

import pytest
import torch

B, T, d, D_I, Hq = 3, 5, 128, 64, 4


@pytest.fixture(scope="module")
def pipeline():
    import __graft_entry__
    __graft_entry__.build()
    from fine_grained_top_b200 import pipeline as m
    return m


def rows(**kw):
    x = dict(q=torch.zeros(B * T, Hq, d), k=torch.zeros(B * T, d), v=torch.zeros(B * T, d), kI=torch.zeros(B * T, D_I),
             n_valid=torch.zeros(B * T, dtype=torch.int32), T=T)
    x.update(kw)
    return x


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(k=torch.zeros(B * T, 2 * d)),            # a projection of keys and values together, contiguous
    dict(v=torch.zeros(B * T, 2 * d)),
    dict(kI=torch.zeros(B * T, 2 * D_I)),
    dict(v=torch.zeros(B * T, d // 2)),
    dict(k=torch.zeros(B * T + 1, d)),            # a row too many
    dict(kI=torch.zeros(B * T - 1, D_I)),         # or too few
    dict(T=1), dict(T=1, q=None),                 # the number of tokens forgotten
    dict(T=T + 1, q=None),
    dict(n_valid=torch.zeros(B, dtype=torch.int32)),
    dict(n_valid=torch.zeros(B * T + 1, dtype=torch.int32)),
])
def test_rows_that_do_not_fit_are_refused(pipeline, q8, bad):
    cache = pipeline.KVCache(B, d, D_I, S_max=256, q8=q8, device="cpu")
    with pytest.raises(ValueError, match="rows"):
        cache.append(**rows(**bad))


def test_rows_that_fit_pass_the_shape_checks(pipeline):
    cache = pipeline.KVCache(B, d, D_I, S_max=256, device="cpu")
    for good in (dict(), dict(k=torch.zeros(B, T, d)), dict(v=torch.zeros(B * T, 3 * d)[:, d:2 * d]), dict(kI=None)):
        with pytest.raises(ValueError, match="not on the GPU"):   # the next check: host tensors
            cache.append(**rows(**good))
