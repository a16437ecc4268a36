"""B200-native fine-grained top-K sparse attention.

The compute lives in ``libsa.so`` (C ABI, ``include/sa.h``): hand-written
CUDA for sm_100a.  This module only marshals arguments to it: every entry
point below has the name and the argument order of its C counterpart, takes
torch tensors for device buffers (PyTorch supplies memory and streams), and
raises ``SAError`` when the library returns a non-OK status.  There is no
Python or CPU fallback: importing fails loudly if the library is missing.

``pipeline`` builds the three-stage step (indexer -> top-K -> sparse
attention) out of these calls with preallocated buffers.
"""

from __future__ import annotations

import ctypes
import os
import struct

# SA_LIBRARY may name another build of the same library (e.g. a tuning variant)
LIB_PATH = os.environ.get("SA_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsa.so")

SA_OK, SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED, SA_ERR_CUDA = 0, 1, 2, 3
SA_ERR_TIMEOUT, SA_ERR_INDEX, SA_ERR_WORKSPACE = 4, 5, 6
SA_DEV_INDEX, SA_DEV_ORDER, SA_DEV_TIMEOUT = 0x1, 0x2, 0x4

# Every symbol include/sa.h declares, with its ctypes signature.
_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "sa_status_string": (ctypes.c_char_p, [_i32]),
    "sa_dev_status_decode": (_i32, [_i32]),
    "sa_version": (_i32, []),
    "sa_indexer_scores": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                 _vp, _vp, _i64, _vp, _vp]),
    "sa_indexer_scores_fp8": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _vp, _vp, _i64, _vp, _vp]),
    "sa_convert_e4m3": (_i32, [_vp, _vp, _i64, _vp]),
    "sa_indexer_scores_candidates": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp,
                                            _i64, _vp, _vp]),
    "sa_block_scores_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "sa_indexer_scores_blocks": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _i64,
                                        _vp, _sz, _vp, _vp]),
    "sa_topk_select": (_i32, [_vp, _i64, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _vp]),
    "sa_topk_select_blocks": (_i32, [_vp, _i64, _i32, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "sa_indexer_topk_decode": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32,
                                      _vp, _vp, _vp]),
    "sa_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "sa_sparse_attn_prefill": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp,
                                      _vp, _vp, _sz, _vp, _vp]),
    "sa_decode_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "sa_sparse_attn_decode": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32,
                                     _i32, _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp, _vp]),
    "sa_sparse_attn_decode_noalloc": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _i32,
                                             _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp, _vp]),
    "sa_cache_append": (_i32, [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                               _i32, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "sa_cache_append_q8": (_i32, [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                                  _i32, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                  _vp, _vp]),
    "sa_sparse_attn_q8": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32,
                                 _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp, _vp]),
    "sa_call": (_i32, [_i32, ctypes.c_char_p, _i32]),
    "sa_pool_index_keys": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "sa_coarse_block_counts": (_i32, [_i32, _i32, _i32, _vp, _vp]),
    "sa_expand_blocks": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp]),
    "sa_selftest_wait_timeout": (_i32, [_i32, _vp, _vp]),
    "sa_selftest_attn_q8_timeout": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _f32, _vp, _i32, _i32, _i32, _vp,
                                           _vp]),
}


class SAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s returned %s" % (where, _lib.sa_status_string(status).decode()))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libsa.so is not built; run `python fine_grained_top_b200/build.py` "
                          "(there is no fallback path)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load()


def _ptr(t):
    """Device (or host) address of a tensor; None -> NULL."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libsa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, where):
    if status != SA_OK:
        raise SAError(status, where)


# ---------------------------------------------------------------- entry points
def sa_indexer_scores(qI, w, kI, page_table, max_pages, pool_pages, page_size, B, T, S, H_I, D_I,
                      n_valid, scores, ld_scores, dev_status=None, stream=None):
    _check(_lib.sa_indexer_scores(_ptr(qI), _ptr(w), _ptr(kI), _ptr(page_table), max_pages, pool_pages,
                                  page_size, B, T, S, H_I, D_I, _ptr(n_valid), _ptr(scores), ld_scores,
                                  _ptr(dev_status), _stream(stream)), "sa_indexer_scores")


def sa_indexer_scores_fp8(qI, w, kI, page_table, max_pages, pool_pages, page_size, B, T, S, H_I, D_I,
                          n_valid, scores, ld_scores, dev_status=None, stream=None):
    """qI, kI: uint8 tensors of e4m3 bits (see sa_convert_e4m3)."""
    _check(_lib.sa_indexer_scores_fp8(_ptr(qI), _ptr(w), _ptr(kI), _ptr(page_table), max_pages, pool_pages,
                                      page_size, B, T, S, H_I, D_I, _ptr(n_valid), _ptr(scores), ld_scores,
                                      _ptr(dev_status), _stream(stream)), "sa_indexer_scores_fp8")


def sa_convert_e4m3(src, dst, n, stream=None):
    _check(_lib.sa_convert_e4m3(_ptr(src), _ptr(dst), n, _stream(stream)), "sa_convert_e4m3")


def sa_indexer_scores_candidates(qI, w, kI, T, S, H_I, D_I, cand, ld_cand, n_cand, scores, ld_scores,
                                 dev_status=None, stream=None):
    _check(_lib.sa_indexer_scores_candidates(_ptr(qI), _ptr(w), _ptr(kI), T, S, H_I, D_I, _ptr(cand),
                                             ld_cand, _ptr(n_cand), _ptr(scores), ld_scores,
                                             _ptr(dev_status), _stream(stream)),
           "sa_indexer_scores_candidates")


def sa_block_scores_workspace_bytes(T, S, keep) -> int:
    return int(_lib.sa_block_scores_workspace_bytes(T, S, keep))


def sa_indexer_scores_blocks(qI, w, kI, T, S, H_I, D_I, blocks, keep, block, scores, ld_scores, workspace,
                             workspace_bytes, dev_status=None, stream=None):
    _check(_lib.sa_indexer_scores_blocks(_ptr(qI), _ptr(w), _ptr(kI), T, S, H_I, D_I, _ptr(blocks), keep, block,
                                         _ptr(scores), ld_scores, _ptr(workspace), workspace_bytes,
                                         _ptr(dev_status), _stream(stream)), "sa_indexer_scores_blocks")


def sa_topk_select(scores, ld_scores, rows, row_len, n_valid, cand_map, ld_cand, K, topk,
                   dev_status=None, stream=None):
    _check(_lib.sa_topk_select(_ptr(scores), ld_scores, rows, row_len, _ptr(n_valid), _ptr(cand_map),
                               ld_cand, K, _ptr(topk), _ptr(dev_status), _stream(stream)), "sa_topk_select")


def sa_topk_select_blocks(scores, ld_scores, T, S, blocks, keep, block, K, topk, dev_status=None, stream=None):
    _check(_lib.sa_topk_select_blocks(_ptr(scores), ld_scores, T, S, _ptr(blocks), keep, block, K, _ptr(topk),
                                      _ptr(dev_status), _stream(stream)), "sa_topk_select_blocks")


def sa_indexer_topk_decode(qI, w, kI, page_table, max_pages, pool_pages, page_size, B, S, H_I, D_I, seq_lens, K,
                           topk, dev_status=None, stream=None):
    _check(_lib.sa_indexer_topk_decode(_ptr(qI), _ptr(w), _ptr(kI), _ptr(page_table), max_pages, pool_pages,
                                       page_size, B, S, H_I, D_I, _ptr(seq_lens), K, _ptr(topk),
                                       _ptr(dev_status), _stream(stream)), "sa_indexer_topk_decode")


def sa_prefill_workspace_bytes(T, S, K, W, Hq, d) -> int:
    return int(_lib.sa_prefill_workspace_bytes(T, S, K, W, Hq, d))


def sa_sparse_attn_prefill(q, k, v, topk, K, W, T, S, Hq, d, scale, out, lse=None, workspace=None,
                           workspace_bytes=0, dev_status=None, stream=None):
    _check(_lib.sa_sparse_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(topk), K, W, T, S, Hq, d,
                                       float(scale), _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                       _ptr(dev_status), _stream(stream)), "sa_sparse_attn_prefill")


def sa_decode_workspace_bytes(B, Hq, d, K, W) -> int:
    return int(_lib.sa_decode_workspace_bytes(B, Hq, d, K, W))


def sa_sparse_attn_decode(q, k_cache, v_cache, page_table, max_pages, pool_pages, page_size, S_max, seq_lens,
                          topk, K, W, B, Hq, d, scale, out, lse, workspace, workspace_bytes,
                          dev_status=None, stream=None):
    _check(_lib.sa_sparse_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), max_pages,
                                      pool_pages, page_size, S_max, _ptr(seq_lens), _ptr(topk), K, W, B,
                                      Hq, d, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                      workspace_bytes, _ptr(dev_status), _stream(stream)),
           "sa_sparse_attn_decode")


def sa_sparse_attn_decode_noalloc(q, k_cache, v_cache, page_table, max_pages, pool_pages, page_size, S_max,
                                  seq_lens, topk, K, W, B, Hq, d, scale, out, lse=None, dev_status=None,
                                  stream=None):
    """Decode for callers that cannot allocate device memory: the split partials
    go to a fixed 16 MiB array inside the library instead of a workspace.
    Concurrent calls on one GPU share that array and must not overlap."""
    _check(_lib.sa_sparse_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                              max_pages, pool_pages, page_size, S_max, _ptr(seq_lens),
                                              _ptr(topk), K, W, B, Hq, d, float(scale), _ptr(out), _ptr(lse),
                                              _ptr(dev_status), _stream(stream)),
           "sa_sparse_attn_decode_noalloc")


SA_DECODE_NOALLOC_SCRATCH_BYTES = 16 << 20


# The entry points of the caches, below, sit between a step's small kernels,
# so what a call costs on the host counts: their checks are one expression, and
# the arguments go over as one array of words (sa_call) instead of one by one.
_T = None                       # torch's types, looked up at the first call that needs them
_CACHE_APPEND, _CACHE_APPEND_Q8, _SPARSE_ATTN_Q8 = 0, 1, 2
_APPEND_WORDS, _APPEND_Q8_WORDS = struct.Struct("29q"), struct.Struct("32q")
_ATTN_Q8_WORDS = struct.Struct("19qd4q")


class _Types:
    def __init__(self):
        import torch
        self.bf, self.i32, self.f32 = torch.bfloat16, torch.int32, torch.float32
        self.f8 = (torch.uint8, torch.float8_e4m3fn)
        self.device, self.current_device = torch.cuda.device, torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _types():
    global _T
    if _T is None:
        _T = _Types()
    return _T


def _refuse(dev, tensors):
    """Raise for the first of (name, tensor, dtypes, least number of elements) that is not a contiguous tensor of one of
    the types on GPU `dev`: a host tensor, or a short one, never reaches a kernel."""
    for name, t, dtypes, numel in tensors:
        dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
        if t is None:
            continue
        if dev < 0 or t.get_device() != dev:
            raise ValueError("%s is not on the GPU of the other tensors" % name)
        if t.dtype not in dtypes or t.numel() < numel or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of at least %d elements"
                             % (name, " or ".join(map(str, dtypes)), numel))


def _rows_at(t, name, dev, bf, n, width, ld):
    """The address of n rows of `width` bf16 values, `ld` apart: contiguous, or a slice [n, width] of wider rows."""
    if t is None:
        return 0
    if t.get_device() != dev or dev < 0:
        raise ValueError("%s is not on the GPU of the other tensors" % name)
    if t.dtype is not bf or n > 0 and (
            t.numel() < (n - 1) * ld + width if t.is_contiguous() else
            t.dim() != 2 or t.shape[0] < n or t.shape[1] < width or t.stride(1) != 1 or t.stride(0) != ld):
        raise ValueError("%s does not hold %d rows of %d bf16 values, %d apart" % (name, n, width, ld))
    return t.data_ptr()


def _call(where, entry, dev, words):
    """The C call on the tensors' GPU."""
    if dev == _T.current_device():
        status = _lib.sa_call(entry, words, len(words) // 8)
    else:
        with _T.device(dev):
            status = _lib.sa_call(entry, words, len(words) // 8)
    if status != SA_OK:
        raise SAError(status, where)


def sa_cache_append(q, ld_q, q_out, k, ld_k, v, ld_v, kI, ld_kI, n_valid, page_table, max_pages, pool_pages, page_size,
                    S_max, B, T, Hq, d, D_I, inv_freq, rot_dim, interleaved, k_cache, v_cache, kI_cache, kI_e4m3,
                    dev_status=None, stream=None):
    """Append the rotated keys and the values of new tokens to a bf16 cache (and
    the index keys to theirs), and rotate the queries.  q, k, v and kI may be
    slices of wider rows (ld_* elements apart)."""
    t = _types()
    bf, i32, R, n, dev = t.bf, t.i32, B * T, pool_pages * 64 if page_table is not None else B * S_max, k_cache.get_device()
    if not (dev >= 0 and k_cache.dtype is bf and k_cache.numel() >= n * d and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype is bf and v_cache.numel() >= n * d and v_cache.is_contiguous()
            and _cache_tensors_ok(t, dev, R, n, q_out, Hq * d, n_valid, page_table, B * max_pages, inv_freq, rot_dim,
                                  kI_cache, kI_e4m3, D_I, dev_status)):
        _refuse(dev, (("k_cache", k_cache, bf, n * d), ("v_cache", v_cache, bf, n * d))
                + _append_tensors(t, R, n, q_out, Hq * d, n_valid, page_table, B * max_pages, inv_freq, rot_dim, kI_cache,
                                  kI_e4m3, D_I, dev_status))
    _call("sa_cache_append", _CACHE_APPEND, dev, _APPEND_WORDS.pack(
        _rows_at(q, "q", dev, bf, R, Hq * d, ld_q), ld_q, _addr(q_out), _rows_at(k, "k", dev, bf, R, d, ld_k), ld_k,
        _rows_at(v, "v", dev, bf, R, d, ld_v), ld_v, _rows_at(kI, "kI", dev, bf, R, D_I, ld_kI), ld_kI, n_valid.data_ptr(),
        _addr(page_table), max_pages, pool_pages, page_size, S_max, B, T, Hq, d, D_I, _addr(inv_freq), rot_dim, interleaved,
        k_cache.data_ptr(), v_cache.data_ptr(), _addr(kI_cache), kI_e4m3, _addr(dev_status),
        t.raw_stream(dev) if stream is None else stream.cuda_stream))


def sa_cache_append_q8(q, ld_q, q_out, k, ld_k, v, ld_v, kI, ld_kI, n_valid, page_table, max_pages, pool_pages, page_size,
                       S_max, B, T, Hq, d, D_I, inv_freq, rot_dim, interleaved, k_cache, v_cache, k_scale, v_scale,
                       scale_block, kI_cache, kI_e4m3, dev_status=None, stream=None):
    """The same append into an 8-bit cache (uint8 or float8_e4m3fn tensors) with a scale for each scale_block tokens."""
    t = _types()
    bf, f8, f32, R, n, dev = t.bf, t.f8, t.f32, B * T, pool_pages * 64 if page_table is not None else B * S_max, k_cache.get_device()
    ns = n // max(scale_block, 1)
    if not (dev >= 0 and k_cache.dtype in f8 and k_cache.numel() >= n * d and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype in f8 and v_cache.numel() >= n * d and v_cache.is_contiguous()
            and k_scale.get_device() == dev and k_scale.dtype is f32 and k_scale.numel() >= ns and k_scale.is_contiguous()
            and v_scale.get_device() == dev and v_scale.dtype is f32 and v_scale.numel() >= ns and v_scale.is_contiguous()
            and _cache_tensors_ok(t, dev, R, n, q_out, Hq * d, n_valid, page_table, B * max_pages, inv_freq, rot_dim,
                                  kI_cache, kI_e4m3, D_I, dev_status)):
        _refuse(dev, (("k_cache", k_cache, f8, n * d), ("v_cache", v_cache, f8, n * d), ("k_scale", k_scale, f32, ns),
                      ("v_scale", v_scale, f32, ns))
                + _append_tensors(t, R, n, q_out, Hq * d, n_valid, page_table, B * max_pages, inv_freq, rot_dim, kI_cache,
                                  kI_e4m3, D_I, dev_status))
    _call("sa_cache_append_q8", _CACHE_APPEND_Q8, dev, _APPEND_Q8_WORDS.pack(
        _rows_at(q, "q", dev, bf, R, Hq * d, ld_q), ld_q, _addr(q_out), _rows_at(k, "k", dev, bf, R, d, ld_k), ld_k,
        _rows_at(v, "v", dev, bf, R, d, ld_v), ld_v, _rows_at(kI, "kI", dev, bf, R, D_I, ld_kI), ld_kI, n_valid.data_ptr(),
        _addr(page_table), max_pages, pool_pages, page_size, S_max, B, T, Hq, d, D_I, _addr(inv_freq), rot_dim, interleaved,
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), scale_block, _addr(kI_cache), kI_e4m3,
        _addr(dev_status), t.raw_stream(dev) if stream is None else stream.cuda_stream))


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _append_tensors(t, R, n, q_out, q_width, n_valid, page_table, pages, inv_freq, rot_dim, kI_cache, kI_e4m3, D_I, dev_status):
    return (("q_out", q_out, t.bf, R * q_width), ("n_valid", n_valid, t.i32, R), ("page_table", page_table, t.i32, pages),
            ("inv_freq", inv_freq, t.f32, rot_dim // 2), ("kI_cache", kI_cache, t.f8 if kI_e4m3 else t.bf, n * D_I),
            ("dev_status", dev_status, t.i32, 1))


def _cache_tensors_ok(t, dev, R, n, q_out, q_width, n_valid, page_table, pages, inv_freq, rot_dim, kI_cache, kI_e4m3, D_I,
                      dev_status):
    """Whether _append_tensors hold, at once."""
    i32 = t.i32
    return (n_valid.get_device() == dev and n_valid.dtype is i32 and n_valid.numel() >= R and n_valid.is_contiguous()
            and (q_out is None or q_out.get_device() == dev and q_out.dtype is t.bf and q_out.numel() >= R * q_width
                 and q_out.is_contiguous())
            and (page_table is None or page_table.get_device() == dev and page_table.dtype is i32
                 and page_table.numel() >= pages and page_table.is_contiguous())
            and (inv_freq is None or inv_freq.get_device() == dev and inv_freq.dtype is t.f32
                 and inv_freq.numel() >= rot_dim // 2 and inv_freq.is_contiguous())
            and (kI_cache is None or kI_cache.get_device() == dev and kI_cache.numel() >= n * D_I and kI_cache.is_contiguous()
                 and (kI_cache.dtype in t.f8 if kI_e4m3 else kI_cache.dtype is t.bf))
            and (dev_status is None or dev_status.get_device() == dev and dev_status.dtype is i32
                 and dev_status.numel() >= 1))


def sa_sparse_attn_q8(q, k_cache, v_cache, k_scale, v_scale, scale_block, page_table, max_pages, pool_pages, page_size,
                      S_max, n_valid, topk, K, W, B, T, Hq, d, scale, out, lse=None, dev_status=None, stream=None):
    """Selected-key attention over an 8-bit cache, T rows a sequence."""
    t = _types()
    R, n, dev = B * T, pool_pages * 64 if page_table is not None else B * S_max, q.get_device()
    bf, f8, f32, i32, ns = t.bf, t.f8, t.f32, t.i32, n // max(scale_block, 1)
    if not (dev >= 0 and q.dtype is bf and q.numel() >= R * Hq * d and q.is_contiguous()
            and k_cache.get_device() == dev and k_cache.dtype in f8 and k_cache.numel() >= n * d and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype in f8 and v_cache.numel() >= n * d and v_cache.is_contiguous()
            and k_scale.get_device() == dev and k_scale.dtype is f32 and k_scale.numel() >= ns and k_scale.is_contiguous()
            and v_scale.get_device() == dev and v_scale.dtype is f32 and v_scale.numel() >= ns and v_scale.is_contiguous()
            and n_valid.get_device() == dev and n_valid.dtype is i32 and n_valid.numel() >= R and n_valid.is_contiguous()
            and out.get_device() == dev and out.dtype is bf and out.numel() >= R * Hq * d and out.is_contiguous()
            and (topk is None or topk.get_device() == dev and topk.dtype is i32 and topk.numel() >= R * K
                 and topk.is_contiguous())
            and (page_table is None or page_table.get_device() == dev and page_table.dtype is i32
                 and page_table.numel() >= B * max_pages and page_table.is_contiguous())
            and (lse is None or lse.get_device() == dev and lse.dtype is f32 and lse.numel() >= R * Hq and lse.is_contiguous())
            and (dev_status is None or dev_status.get_device() == dev and dev_status.dtype is i32
                 and dev_status.numel() >= 1)):
        _refuse(dev, (("q", q, bf, R * Hq * d), ("k_cache", k_cache, f8, n * d), ("v_cache", v_cache, f8, n * d),
                      ("k_scale", k_scale, f32, ns), ("v_scale", v_scale, f32, ns), ("n_valid", n_valid, i32, R),
                      ("out", out, bf, R * Hq * d), ("topk", topk, i32, R * K), ("page_table", page_table, i32, B * max_pages),
                      ("lse", lse, f32, R * Hq), ("dev_status", dev_status, i32, 1)))
    _call("sa_sparse_attn_q8", _SPARSE_ATTN_Q8, dev, _ATTN_Q8_WORDS.pack(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), scale_block,
        _addr(page_table), max_pages, pool_pages, page_size, S_max, n_valid.data_ptr(), _addr(topk), K, W, B, T, Hq, d, scale,
        out.data_ptr(), _addr(lse), _addr(dev_status), t.raw_stream(dev) if stream is None else stream.cuda_stream))


def sa_pool_index_keys(kI, S, D_I, block, kB, stream=None):
    _check(_lib.sa_pool_index_keys(_ptr(kI), S, D_I, block, _ptr(kB), _stream(stream)), "sa_pool_index_keys")


def sa_coarse_block_counts(T, S, block, n_blocks, stream=None):
    _check(_lib.sa_coarse_block_counts(T, S, block, _ptr(n_blocks), _stream(stream)), "sa_coarse_block_counts")


def sa_expand_blocks(blocks, T, S, keep, block, cand, ld_cand, n_cand, dev_status=None, stream=None):
    _check(_lib.sa_expand_blocks(_ptr(blocks), T, S, keep, block, _ptr(cand), ld_cand, _ptr(n_cand),
                                 _ptr(dev_status), _stream(stream)), "sa_expand_blocks")


def sa_dev_status_decode(word: int) -> int:
    return int(_lib.sa_dev_status_decode(int(word)))


def sa_version() -> int:
    return int(_lib.sa_version())


def sa_selftest_attn_q8_timeout(q, k_cache, v_cache, k_scale, v_scale, S_max, n_valid, B, Hq, scale, out, ctas, lost,
                                limit_us, dev_status, stream=None):
    t, n = _types(), B * S_max
    bf, dev = t.bf, q.get_device()
    _refuse(dev, (("q", q, bf, B * Hq * 128), ("k_cache", k_cache, t.f8, n * 128), ("v_cache", v_cache, t.f8, n * 128),
                  ("k_scale", k_scale, t.f32, n // 64), ("v_scale", v_scale, t.f32, n // 64), ("n_valid", n_valid, t.i32, B),
                  ("out", out, bf, B * Hq * 128), ("dev_status", dev_status, t.i32, 1)))
    _check(_lib.sa_selftest_attn_q8_timeout(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), S_max,
                                            _ptr(n_valid), B, Hq, scale, _ptr(out), ctas, lost, int(limit_us),
                                            _ptr(dev_status), _stream(stream)), "sa_selftest_attn_q8_timeout")


def sa_selftest_wait_timeout(limit_us, dev_status, stream=None):
    _check(_lib.sa_selftest_wait_timeout(int(limit_us), _ptr(dev_status), _stream(stream)),
           "sa_selftest_wait_timeout")
