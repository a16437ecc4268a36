"""Argument checks and host logic of the cache append and the 8-bit cache's
attention (no GPU: the checks run before any CUDA call)."""

import ctypes
import struct

import pytest
import torch

from tests.conftest import ROOT  # noqa: F401


@pytest.fixture(scope="module")
def sa():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_top_b200 as m
    return m


P = ctypes.c_void_p(256)   # a fake, aligned, never dereferenced pointer
ODD = ctypes.c_void_p(264)


def append_args(**kw):
    a = dict(q=P, ld_q=2048, q_out=ctypes.c_void_p(4096), k=P, ld_k=128, v=P, ld_v=128, kI=P, ld_kI=64, n_valid=P,
             page_table=None, max_pages=0, pool_pages=0, page_size=64, S_max=1024, B=2, T=3, Hq=16, d=128, D_I=64,
             inv_freq=P, rot_dim=128, interleaved=0, k_cache=P, v_cache=P)
    tail = dict(kI_cache=P, kI_e4m3=0, dev_status=None, stream=None)
    scales = dict(k_scale=P, v_scale=P, scale_block=64)
    q8 = kw.pop("q8", False)
    for name, value in kw.items():
        (a if name in a else tail if name in tail else scales)[name] = value
    return list(a.values()) + (list(scales.values()) if q8 else []) + list(tail.values())


BAD_APPEND = [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(Hq=65), "UNSUPPORTED"),
    (dict(Hq=0), "UNSUPPORTED"), (dict(rot_dim=24), "UNSUPPORTED"), (dict(rot_dim=144), "UNSUPPORTED"),
    (dict(rot_dim=-16), "UNSUPPORTED"), (dict(D_I=48), "UNSUPPORTED"), (dict(q=None), "INVALID_ARG"),
    (dict(q_out=None), "INVALID_ARG"), (dict(kI=None), "INVALID_ARG"), (dict(kI_cache=None), "INVALID_ARG"),
    (dict(k=None), "INVALID_ARG"), (dict(v_cache=None), "INVALID_ARG"), (dict(n_valid=None), "INVALID_ARG"),
    (dict(inv_freq=None), "INVALID_ARG"), (dict(ld_q=2040), "INVALID_ARG"), (dict(ld_k=132), "INVALID_ARG"),
    (dict(ld_v=64), "INVALID_ARG"), (dict(ld_kI=32), "INVALID_ARG"), (dict(k=ODD), "INVALID_ARG"),
    (dict(k_cache=ODD), "INVALID_ARG"), (dict(q_out=P, ld_q=4096), "INVALID_ARG"),   # in place in wider rows
    (dict(S_max=-64), "INVALID_ARG"), (dict(B=40000, S_max=65536), "UNSUPPORTED"),
    (dict(page_table=P, max_pages=16, pool_pages=40, page_size=32), "UNSUPPORTED"),
    (dict(page_table=P, max_pages=0, pool_pages=40), "INVALID_ARG"),
    (dict(page_table=P, max_pages=16, pool_pages=0), "INVALID_ARG"),
    (dict(page_table=P, max_pages=16, pool_pages=1 << 25), "UNSUPPORTED"),
    (dict(B=0), "OK"), (dict(T=0), "OK"),
]


@pytest.mark.parametrize("kw,want", BAD_APPEND)
@pytest.mark.parametrize("q8", [False, True])
def test_append_refusals(sa, kw, want, q8):
    f = sa._lib.sa_cache_append_q8 if q8 else sa._lib.sa_cache_append
    code = sa.SA_OK if want == "OK" else getattr(sa, "SA_ERR_" + want)
    assert f(*append_args(q8=q8, **kw)) == code


@pytest.mark.parametrize("kw,want", [
    (dict(scale_block=0), "UNSUPPORTED"), (dict(scale_block=48), "UNSUPPORTED"), (dict(scale_block=128), "UNSUPPORTED"),
    (dict(S_max=1000), "INVALID_ARG"), (dict(k_scale=None), "INVALID_ARG"), (dict(v_scale=None), "INVALID_ARG"),
    (dict(T=131073), "UNSUPPORTED")])
def test_append_q8_refusals(sa, kw, want):
    assert sa._lib.sa_cache_append_q8(*append_args(q8=True, **kw)) == getattr(sa, "SA_ERR_" + want)


def attn_args(**kw):
    a = dict(q=P, k=P, v=P, ks=P, vs=P, scale_block=64, page_table=None, max_pages=0, pool_pages=0, page_size=64, S_max=1024,
             n_valid=P, topk=P, K=64, W=16, B=2, T=3, Hq=16, d=128, scale=0.1, out=P, lse=None, dev_status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(K=-1), "INVALID_ARG"), (dict(W=-1), "INVALID_ARG"), (dict(K=0, W=0), "INVALID_ARG"), (dict(B=-2), "INVALID_ARG"),
    (dict(T=-2), "INVALID_ARG"), (dict(d=32), "UNSUPPORTED"), (dict(Hq=0), "UNSUPPORTED"), (dict(Hq=128), "UNSUPPORTED"),
    (dict(K=524288, W=1), "UNSUPPORTED"), (dict(scale_block=3), "UNSUPPORTED"), (dict(S_max=1001), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(ks=None), "INVALID_ARG"), (dict(topk=None), "INVALID_ARG"),
    (dict(n_valid=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(v=ODD), "INVALID_ARG"),
    (dict(out=ODD), "INVALID_ARG"), (dict(page_table=P, max_pages=4, pool_pages=9, page_size=16), "UNSUPPORTED"),
    (dict(page_table=P, max_pages=4, pool_pages=-1), "INVALID_ARG"), (dict(B=1 << 20, T=1 << 10, S_max=64), "UNSUPPORTED"),
    (dict(B=0), "OK"), (dict(T=0), "OK")])
def test_attention_q8_refusals(sa, kw, want):
    code = sa.SA_OK if want == "OK" else getattr(sa, "SA_ERR_" + want)
    assert sa._lib.sa_sparse_attn_q8(*attn_args(**kw)) == code


def test_calls_by_words(sa):
    """sa_call checks its words and hands them to the same checks as the call itself."""
    f, S = sa._lib.sa_call, struct.Struct("19qd4q")
    a = [0 if v is None else getattr(v, "value", v) for v in attn_args()]
    assert f(2, S.pack(*attn_words(B=0)), 24) == sa.SA_OK
    assert f(2, S.pack(*attn_words(d=32)), 24) == sa.SA_ERR_UNSUPPORTED
    assert f(2, S.pack(*a), 23) == sa.SA_ERR_INVALID_ARG                      # a word short
    assert f(3, S.pack(*a), 24) == sa.SA_ERR_INVALID_ARG                      # no such entry
    assert f(2, None, 24) == sa.SA_ERR_INVALID_ARG
    assert f(2, S.pack(*attn_words(B=2 ** 32)), 24) == sa.SA_ERR_INVALID_ARG   # would be 0 in 32 bits
    w = [0 if v is None else getattr(v, "value", v) for v in append_args(T=0)]
    assert f(0, struct.pack("29q", *w), 29) == sa.SA_OK
    w = [0 if v is None else getattr(v, "value", v) for v in append_args(q8=True, rot_dim=8)]
    assert f(1, struct.pack("32q", *w), 32) == sa.SA_ERR_UNSUPPORTED


def attn_words(**kw):
    return [0 if v is None else getattr(v, "value", v) for v in attn_args(**kw)]


def test_tensors_of_the_wrong_kind_are_refused(sa):
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    z = lambda *s, dtype: torch.zeros(*s, dtype=dtype)  # noqa: E731
    args = [z(2, 4, 64, dtype=bf), z(2, 128, 64, dtype=u8), z(2, 128, 64, dtype=u8), z(2, 2, dtype=f32), z(2, 2, dtype=f32), 64,
            None, 0, 0, 64, 128, z(2, dtype=i32), z(2, 8, dtype=i32), 8, 4, 2, 1, 4, 64, 0.125, z(2, 4, 64, dtype=bf)]
    with pytest.raises(ValueError, match="not on the GPU"):   # host tensors never reach a kernel
        sa.sa_sparse_attn_q8(*args)


def meta(*s, dtype):
    """A tensor that says it is on GPU 0 and has no memory: the checks fail before anything is called."""
    class OnGpu:
        def __init__(self, t):
            self.t, self.dtype = t, t.dtype

        def get_device(self):
            return 0

        def __getattr__(self, n):
            return getattr(self.t, n)
    return OnGpu(torch.zeros(*s, dtype=dtype, device="meta"))


@pytest.mark.parametrize("at,bad", [(0, meta(2, 4, 64, dtype=torch.float32)), (1, meta(2, 128, 64, dtype=torch.bfloat16)),
                                    (3, meta(1, 2, dtype=torch.float32)), (11, meta(2, dtype=torch.int64)),
                                    (12, meta(1, 8, dtype=torch.int32)), (20, meta(2, 4, 32, dtype=torch.bfloat16))])
def test_short_or_mistyped_tensors_are_refused(sa, at, bad):
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    args = [meta(2, 4, 64, dtype=bf), meta(2, 128, 64, dtype=u8), meta(2, 128, 64, dtype=u8), meta(2, 2, dtype=f32),
            meta(2, 2, dtype=f32), 64, None, 0, 0, 64, 128, meta(2, dtype=i32), meta(2, 8, dtype=i32), 8, 4, 2, 1, 4, 64, 0.125,
            meta(2, 4, 64, dtype=bf)]
    args[at] = bad
    with pytest.raises(ValueError):
        sa.sa_sparse_attn_q8(*args)


def test_cache_and_plan_shapes():
    from fine_grained_top_b200 import pipeline
    c = pipeline.KVCache(3, 128, 64, paged=True, max_pages=4, pool_pages=20, q8=True, scale_block=16, device="cpu")
    assert tuple(c.k.shape) == (20, 64, 128) and c.k.dtype == torch.uint8 and tuple(c.k_scale.shape) == (20, 4)
    assert c.S_max == 256 and tuple(c.inv_freq.shape) == (64,) and float(c.inv_freq[0]) == 1.0
    p = pipeline.DecodePlan(3, 16, 128, 4, 64, 64, 32, T=5, cache=c, device="cpu")
    assert p.kv_q8 and p.scale_block == 16 and p.ws_bytes == 0 and tuple(p.topk.shape) == (15, 64)
    assert p.launches() == 4
    names = [n for n, _ in p.stages({k: None for k in ("q", "k", "v", "qI", "w", "kI", "lengths")})]
    assert names == ["append", "indexer", "topk", "attention"]
    b = pipeline.KVCache(2, 64, 32, S_max=100, device="cpu")
    assert tuple(b.k.shape) == (2, 100, 64) and b.k.dtype == torch.bfloat16 and b.k_scale is None
    assert pipeline.DecodePlan(2, 16, 64, 4, 32, 64, 32, cache=b, device="cpu").launches() == 4
    with pytest.raises(ValueError):
        pipeline.KVCache(2, 64, 32, S_max=100, q8=True, scale_block=64, device="cpu")   # blocks cross sequences
    with pytest.raises(ValueError):
        pipeline.DecodePlan(2, 16, 64, 4, 32, 64, 32, S_max=128, T=2, device="cpu")     # bf16 caches: one query
    with pytest.raises(ValueError):
        pipeline.DecodePlan(2, 16, 128, 4, 32, 64, 32, cache=b, device="cpu")           # another head dim
    q, ld = c._rows(torch.zeros(15, 300)[:, 20:148], 15, 128)
    assert ld == 300 and tuple(q.shape) == (15, 128)
    with pytest.raises(ValueError):
        c._rows(torch.zeros(300, 15).T[:, 20:148], 15, 128)
    new = dict(k=torch.zeros(15, 128), v=torch.zeros(15, 128), kI=torch.zeros(15, 64), n_valid=torch.zeros(15), T=5)
    with pytest.raises(ValueError, match="page table"):
        c.append(None, **new)
    with pytest.raises(ValueError, match="whole heads"):
        c.append(torch.zeros(15 * 128 + 8), page_table=torch.zeros(3, 4), **new)
