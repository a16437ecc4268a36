"""The three-stage step built from the C-ABI calls, with buffers allocated once.

A plan owns its intermediate buffers (torch device tensors) and enqueues the
library's kernels on one stream; the host does no arithmetic of the method.

    PrefillPlan    indexer -> top-K -> sparse attention for one causal
                   sequence (optionally the two-stage coarse/fine selection)
    DecodePlan     one new query per sequence over a contiguous or paged
                   KV cache: indexer -> top-K -> split-K attention + merge;
                   over an 8-bit cache also a chunk of T queries per sequence
    KVCache        the caches of B sequences (16 or 8 bits) and the append
                   that fills them with rotated keys, a first stage of a
                   DecodePlan that is given one
    HostPipeline   steps fed from and read back to pinned host memory, the
                   copies of neighbouring steps overlapped with the kernels

``stages(inputs)`` returns the step as a list of (name, launch) pairs, one
per C-ABI call, so that callers can time each kernel; ``run`` executes them.
"""

from __future__ import annotations

import contextlib
import math

import torch

from . import (sa_block_scores_workspace_bytes, sa_cache_append, sa_cache_append_q8, sa_coarse_block_counts,
               sa_decode_workspace_bytes,
               sa_indexer_scores, sa_indexer_scores_blocks, sa_indexer_scores_fp8, sa_indexer_topk_decode,
               sa_pool_index_keys,
               sa_prefill_workspace_bytes, sa_sparse_attn_decode, sa_sparse_attn_prefill,
               sa_sparse_attn_q8, sa_topk_select,
               sa_topk_select_blocks)


def _ld(n: int) -> int:
    return max(4, (n + 3) // 4 * 4)


class PrefillPlan:
    """Buffers for N queries of one causal sequence of S keys (default S = N):
    the queries sit at the last N positions, S - N .. S - 1 (S > N is one
    rank's chunk of a longer sequence, see ``shard``).
    Inputs: dict with q [N,Hq,d], qI [N,H_I,D_I], w [N,H_I] and k/v [S,d],
    kI [S,D_I].
    index_fp8: qI and kI are e4m3 bytes (uint8) and the indexer runs in FP8
    (single-stage selection only)."""

    def __init__(self, N, Hq, d, H_I, D_I, K, W, block=None, keep=None, row_blocks=1, index_fp8=False,
                 device="cuda", S=None):
        if index_fp8 and block is not None:
            raise ValueError("the FP8 indexer serves the single-stage selection")
        S = N if S is None else int(S)
        if S < N:
            raise ValueError("a plan's N queries are the last N of its S keys (S >= N)")
        self.N, self.S, self.Hq, self.d, self.H_I, self.D_I, self.K, self.W = N, S, Hq, d, H_I, D_I, K, W
        self.index = sa_indexer_scores_fp8 if index_fp8 else sa_indexer_scores
        self.block, self.keep = block, keep
        # single-stage only: score and select the queries in row_blocks blocks,
        # so that a block's scores are still in L2 when top-K reads them
        self.row_blocks = max(1, int(row_blocks)) if (block is None and S == N) else 1
        self.scale = 1.0 / math.sqrt(d)
        dev = torch.device(device)
        i32, f32 = torch.int32, torch.float32
        self.topk = torch.empty((N, K), dtype=i32, device=dev)
        self.out = torch.empty((N, Hq, d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((N, Hq), dtype=f32, device=dev)
        self.dev_status = torch.zeros(1, dtype=i32, device=dev)
        # The masked tensor-core attention (selected by passing its bitmap
        # workspace) runs one CTA per 256 query-head rows; below one CTA per SM
        # the gathered kernel is faster.
        groups = N * Hq // 256
        sms = torch.cuda.get_device_properties(dev).multi_processor_count if dev.type == "cuda" else 148
        self.attn_ws_bytes = sa_prefill_workspace_bytes(N, S, K, W, Hq, d) if groups >= sms else 0
        self.attn_ws = (torch.empty(self.attn_ws_bytes, dtype=torch.uint8, device=dev)
                        if self.attn_ws_bytes else None)
        if block is None:
            self.ld = _ld(S)
            self.scores = torch.empty((N, self.ld), dtype=f32, device=dev)
        else:
            self.nb = S // block
            self.ld_coarse = _ld(self.nb)
            self.kB = torch.empty((max(self.nb, 1), D_I), dtype=torch.bfloat16, device=dev)
            self.n_blocks = torch.empty(N, dtype=i32, device=dev)
            self.coarse = torch.empty((N, self.ld_coarse), dtype=f32, device=dev)
            self.blocks = torch.empty((N, keep), dtype=i32, device=dev)
            self.ld_cand = _ld(keep * block + block)
            self.fine = torch.empty((N, self.ld_cand), dtype=f32, device=dev)
            self.ws_bytes = sa_block_scores_workspace_bytes(N, S, keep)
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    def stages(self, x, stream=None):
        N, S, K, ds, H, D = self.N, self.S, self.K, self.dev_status, self.H_I, self.D_I
        attn = ("attention", lambda: sa_sparse_attn_prefill(
            x["q"], x["k"], x["v"], self.topk, K, self.W, N, S, self.Hq, self.d, self.scale, self.out,
            self.lse, self.attn_ws, self.attn_ws_bytes, ds, stream))
        if self.block is None and self.row_blocks > 1:
            # queries t0..t1-1 are the last t1 - t0 of a t1-key causal sequence
            bounds = [N * b // self.row_blocks for b in range(self.row_blocks + 1)]
            out = []
            for b in range(self.row_blocks):
                t0, t1 = bounds[b], bounds[b + 1]
                if t1 <= t0:
                    continue
                out.append(("indexer", lambda t0=t0, t1=t1: self.index(
                    x["qI"][t0:t1], x["w"][t0:t1], x["kI"], None, 0, 0, 64, 1, t1 - t0, t1, H, D, None,
                    self.scores[t0:t1], self.ld, ds, stream)))
                out.append(("topk", lambda t0=t0, t1=t1: sa_topk_select(
                    self.scores[t0:t1], self.ld, t1 - t0, t1, None, None, 0, K, self.topk[t0:t1], ds, stream)))
            return out + [attn]
        if self.block is None:
            return [
                ("indexer", lambda: self.index(x["qI"], x["w"], x["kI"], None, 0, 0, 64, 1, N, S, H, D,
                                               None, self.scores, self.ld, ds, stream)),
                ("topk", lambda: sa_topk_select(self.scores, self.ld, N, S, None, None, 0, K, self.topk, ds,
                                                stream)),
                attn]
        blk, keep = self.block, self.keep
        return [
            ("pool", lambda: sa_pool_index_keys(x["kI"], S, D, blk, self.kB, stream)),
            ("block_counts", lambda: sa_coarse_block_counts(N, S, blk, self.n_blocks, stream)),
            ("coarse_indexer", lambda: sa_indexer_scores(x["qI"], x["w"], self.kB, None, 0, 0, 64, 1, N, self.nb,
                                                         H, D, self.n_blocks, self.coarse, self.ld_coarse, ds,
                                                         stream)),
            ("coarse_topk", lambda: sa_topk_select(self.coarse, self.ld_coarse, N, self.nb, self.n_blocks, None,
                                                   0, keep, self.blocks, ds, stream)),
            ("fine_indexer", lambda: sa_indexer_scores_blocks(x["qI"], x["w"], x["kI"], N, S, H, D, self.blocks,
                                                              keep, blk, self.fine, self.ld_cand, self.workspace,
                                                              self.ws_bytes, ds, stream)),
            ("fine_topk", lambda: sa_topk_select_blocks(self.fine, self.ld_cand, N, S, self.blocks, keep, blk, K,
                                                        self.topk, ds, stream)),
            attn]

    def run(self, q, k, v, qI, w, kI, stream=None):
        for _, fn in self.stages(dict(q=q, k=k, v=v, qI=qI, w=w, kI=kI), stream):
            fn()
        return self.out

    def launches(self) -> int:
        """Kernels one run() enqueues: indexer + top-K (per row block), or for
        the two-stage selection pool, block counts, coarse indexer, coarse
        top-k, the fine scores' invert count / scan / scatter and block
        kernel, and the fine top-K over the kept block ids (9); then the
        attention."""
        attn = 2 if self.attn_ws is not None else 1   # (selection bitmap +) attention
        return (2 * self.row_blocks if self.block is None else 9) + attn


class KVCache:
    """The caches of B sequences: keys and values of the one KV head and index
    keys, contiguous ([B, S_max, *]) or pools of 64-token pages ([pool_pages,
    64, *], addressed by the page table that append() and the plans are given).

    q8: keys and values in e4m3 with one power-of-two scale for each
    scale_block tokens (else bf16); index_fp8: e4m3 index keys.
    Positions: pairs of the first rot_dim dims (default all) turn by
    p * inv_freq[i]; inv_freq defaults to theta^(-2i / rot_dim).
    interleaved: pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2).
    The caches are zeroed on the stream that is current here; an append on
    another waits for it first (stream.wait_stream)."""

    def __init__(self, B, d, D_I, S_max=0, paged=False, max_pages=0, pool_pages=0, q8=False, scale_block=64,
                 index_fp8=False, rot_dim=None, theta=10000.0, inv_freq=None, interleaved=False, device="cuda"):
        self.B, self.d, self.D_I, self.paged, self.q8, self.scale_block = B, d, D_I, paged, q8, scale_block
        self.max_pages, self.pool_pages = (max_pages, pool_pages) if paged else (0, 0)
        self.S_max = max_pages * 64 if paged else S_max
        self.index_fp8, self.interleaved = index_fp8, interleaved
        self.rot_dim = d if rot_dim is None else rot_dim
        if q8 and not (1 <= scale_block <= 64 and scale_block & (scale_block - 1) == 0 and self.S_max % scale_block == 0):
            raise ValueError("scale_block is a power of two up to 64 that divides the cache's length")
        dev = torch.device(device)
        if inv_freq is None:
            i = torch.arange(self.rot_dim // 2, dtype=torch.float64)
            inv_freq = (theta ** (-2 * i / max(self.rot_dim, 1))).float()
        self.inv_freq = inv_freq.to(device=dev, dtype=torch.float32).contiguous()
        if self.inv_freq.numel() < self.rot_dim // 2:
            raise ValueError("inv_freq needs rot_dim / 2 entries")
        lead = (pool_pages, 64) if paged else (B, S_max)
        kv, index = torch.uint8 if q8 else torch.bfloat16, torch.uint8 if index_fp8 else torch.bfloat16
        self.k = torch.zeros(lead + (d,), dtype=kv, device=dev)
        self.v = torch.zeros(lead + (d,), dtype=kv, device=dev)
        self.kI = torch.zeros(lead + (D_I,), dtype=index, device=dev)
        self.k_scale = self.v_scale = None
        if q8:
            blocks = (lead[0], lead[1] // scale_block)
            self.k_scale = torch.ones(blocks, dtype=torch.float32, device=dev)
            self.v_scale = torch.ones(blocks, dtype=torch.float32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    @staticmethod
    def _rows(t, R, width):
        """(tensor, row stride) of R rows of `width` values: contiguous, or slices of wider rows."""
        if t is None:
            return None, 0
        if t.is_contiguous():
            if t.numel() != R * width:   # rows of another width, or another number of them
                raise ValueError("%d values where %d rows of %d are new" % (t.numel(), R, width))
            return t, width
        if t.dim() != 2 or tuple(t.shape) != (R, width) or t.stride(1) != 1:
            raise ValueError("new rows are contiguous, or [rows, %d] slices of wider rows" % width)
        return t, t.stride(0)

    def append(self, q, k, v, kI, n_valid, T=1, page_table=None, q_out=None, stream=None, dev_status=None):
        """Write the new tokens' rotated keys, values and index keys ([B*T, *])
        to their slots (row b*T + t at position n_valid[b*T + t] - 1, 0:
        padding) and return the rotated queries (q [B*T, Hq, d], q_out or a new
        tensor of `stream`; None when q is None)."""
        R, d = self.B * T, self.d
        if self.paged and page_table is None:
            raise ValueError("a paged cache is appended to through its page table")
        if n_valid.numel() != R:
            raise ValueError("n_valid has %d entries where %d rows are new" % (n_valid.numel(), R))
        Hq = q.numel() // (R * d) if q is not None and R > 0 else 1
        if q is not None and q.numel() != R * Hq * d:
            raise ValueError("q holds whole heads of %d values for each of %d rows" % (d, R))
        if q is not None and q_out is None:
            # on the stream that writes it: zeros of another could land after the kernel
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                q_out = torch.zeros((R, Hq, d), dtype=torch.bfloat16, device=q.device)
        (q, ld_q), (k, ld_k) = self._rows(q, R, Hq * d), self._rows(k, R, d)
        (v, ld_v), (kI, ld_kI) = self._rows(v, R, d), self._rows(kI, R, self.D_I)
        status = self.dev_status if dev_status is None else dev_status
        rows = (q, ld_q, q_out, k, ld_k, v, ld_v, kI, ld_kI, n_valid, page_table if self.paged else None, self.max_pages,
                self.pool_pages, 64, self.S_max, self.B, T, Hq, d, self.D_I, self.inv_freq, self.rot_dim,
                int(self.interleaved), self.k, self.v)
        index = (self.kI if kI is not None else None, int(self.index_fp8), status, stream)
        if self.q8:
            sa_cache_append_q8(*rows, self.k_scale, self.v_scale, self.scale_block, *index)
        else:
            sa_cache_append(*rows, *index)
        return q_out


class DecodePlan:
    """Buffers for B sequences, one query each, over a contiguous ([B, S_max, *])
    or paged (pools [P, 64, *] + page_table [B, max_pages]) cache.
    Inputs: dict with q [B,Hq,d], k/v/kI caches, qI [B,H_I,D_I], w [B,H_I],
    lengths [B] int32 and, when paged, page_table.
    index_fp8: the qI and kI cache hold e4m3 bytes (uint8); FP8 indexer.
    kv_q8: k and v are 8-bit caches (uint8) and the inputs hold k_scale and
    v_scale too, one for each scale_block tokens; T queries per sequence (rows
    b*T + t of q, qI and w), and lengths [B*T] gives the cached tokens that each
    of them sees (0: padding).
    cache: a KVCache.  Each step then begins by appending its tokens: the inputs
    k, v and kI are the new tokens' rows [B*T, *] and q is not yet rotated; kv_q8,
    scale_block, index_fp8 (for kI; qI is e4m3 too then) and the cache's sizes
    are taken from it."""

    def __init__(self, B, Hq, d, H_I, D_I, K, W, S_max=0, paged=False, max_pages=0, pool_pages=0,
                 index_fp8=False, fused=None, device="cuda", kv_q8=False, scale_block=64, T=1, cache=None):
        if cache is not None:
            if (cache.B, cache.d, cache.D_I) != (B, d, D_I):
                raise ValueError("the cache holds other sequences or dims than the plan")
            paged, max_pages, pool_pages, S_max = cache.paged, cache.max_pages, cache.pool_pages, cache.S_max
            kv_q8, scale_block, index_fp8 = cache.q8, cache.scale_block, cache.index_fp8
        if T != 1 and not kv_q8:
            raise ValueError("several queries per sequence need the 8-bit cache's attention (kv_q8)")
        if T < 1:
            raise ValueError("a step has at least one query per sequence")
        self.kv_q8, self.scale_block, self.T, self.cache = kv_q8, scale_block, T, cache
        self.B, self.Hq, self.d, self.H_I, self.D_I, self.K, self.W = B, Hq, d, H_I, D_I, K, W
        self.index = sa_indexer_scores_fp8 if index_fp8 else sa_indexer_scores
        self.paged, self.max_pages, self.pool_pages = paged, max_pages, pool_pages
        self.S = max_pages * 64 if paged else S_max
        self.S_max = S_max
        # fused=True: indexer and top-K in one kernel (the scores never leave
        # shared memory).  It takes bf16 operands, H_I <= 8, D_I in (64, 128)
        # and rows of at most 262144 keys.  It is not the default: on the
        # decode workloads the two kernels apart are faster (the fused kernel
        # holds one CTA per SM for the whole select, so its key reads run at
        # about half the separate indexer's rate).
        fusable = not index_fp8 and H_I <= 8 and D_I in (64, 128) and self.S <= 262144
        self.fused = False if fused is None else bool(fused)
        if self.fused and T != 1:
            raise ValueError("the fused indexer + top-K takes one query per sequence")
        if self.fused and not fusable:
            raise ValueError("the fused indexer + top-K takes bf16 operands, H_I <= 8, D_I in (64, 128) and "
                             "rows of at most 262144 keys")
        self.scale = 1.0 / math.sqrt(d)
        dev = torch.device(device)
        R = B * T
        self.ld = _ld(self.S)
        self.scores = None if self.fused else torch.empty((R, self.ld), dtype=torch.float32, device=dev)
        self.topk = torch.empty((R, K), dtype=torch.int32, device=dev)
        self.out = torch.empty((R, Hq, d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((R, Hq), dtype=torch.float32, device=dev)
        self.q_rot = torch.zeros((R, Hq, d), dtype=torch.bfloat16, device=dev) if cache is not None else None
        self.ws_bytes = 0 if kv_q8 else sa_decode_workspace_bytes(B, Hq, d, K, W)   # the 8-bit attention has none
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    def stages(self, x, stream=None):
        ds, pt = self.dev_status, x.get("page_table")
        append = []
        if self.cache is not None:
            c, new = self.cache, x
            append = [("append", lambda: c.append(new["q"], new["k"], new["v"], new["kI"], new["lengths"], self.T, pt,
                                                  self.q_rot, stream, ds))]
            x = dict(x, q=self.q_rot, k=c.k, v=c.v, kI=c.kI, k_scale=c.k_scale, v_scale=c.v_scale)
        if self.fused:
            select = [("indexer_topk", lambda: sa_indexer_topk_decode(
                x["qI"], x["w"], x["kI"], pt, self.max_pages, self.pool_pages, 64, self.B, self.S, self.H_I,
                self.D_I, x["lengths"], self.K, self.topk, ds, stream))]
        else:
            select = [
                ("indexer", lambda: self.index(x["qI"], x["w"], x["kI"], pt, self.max_pages, self.pool_pages,
                                               64, self.B, self.T, self.S, self.H_I, self.D_I, x["lengths"],
                                               self.scores, self.ld, ds, stream)),
                ("topk", lambda: sa_topk_select(self.scores, self.ld, self.B * self.T, self.S, x["lengths"], None, 0,
                                                self.K, self.topk, ds, stream))]
        if self.kv_q8:
            attention = ("attention", lambda: sa_sparse_attn_q8(
                x["q"], x["k"], x["v"], x["k_scale"], x["v_scale"], self.scale_block, pt, self.max_pages,
                self.pool_pages, 64, self.S_max, x["lengths"], self.topk, self.K, self.W, self.B, self.T, self.Hq,
                self.d, self.scale, self.out, self.lse, ds, stream))
        else:
            attention = ("attention", lambda: sa_sparse_attn_decode(
                x["q"], x["k"], x["v"], pt, self.max_pages, self.pool_pages, 64, self.S_max, x["lengths"],
                self.topk, self.K, self.W, self.B, self.Hq, self.d, self.scale, self.out, self.lse,
                self.workspace, self.ws_bytes, ds, stream))
        return append + select + [attention]

    def run(self, q, k_cache, v_cache, qI, w, kI, seq_lens, page_table=None, stream=None, k_scale=None, v_scale=None):
        x = dict(q=q, k=k_cache, v=v_cache, qI=qI, w=w, kI=kI, lengths=seq_lens, page_table=page_table,
                 k_scale=k_scale, v_scale=v_scale)
        for _, fn in self.stages(x, stream):
            fn()
        return self.out

    def launches(self) -> int:
        """Kernels one run() enqueues: the fused indexer + top-K (or, unfused,
        the indexer and the top-K), then the attention of
        sa_sparse_attn_decode.  That is one kernel when a thread-block cluster
        of G = min(16, max(1, ceil((K+W)/128), ceil(Hq/8))) CTAs per sequence
        leaves each CTA at most 1024 keys (partials merged in distributed
        shared memory), else a split-K kernel and a merge kernel.  The 8-bit
        cache's attention is always one kernel; a plan with a cache appends
        in one more."""
        if self.kv_q8:
            return (1 if self.fused else 2) + 1 + (self.cache is not None)
        kw = self.K + self.W
        G = min(16, max(1, -(-kw // 128), -(-self.Hq // 8)))
        return (1 if self.fused else 2) + (1 if -(-kw // G) <= 1024 else 2) + (self.cache is not None)


class HostPipeline:
    """Steps whose inputs come from pinned host memory and whose output goes
    back to pinned host memory, with the copies running under the kernels.

    Two plans (two sets of device buffers) alternate.  Step i uploads its
    inputs into set i % 2 on an upload stream, runs the path on the compute
    stream and downloads the plan's output on a download stream.  Its upload
    waits only for step i - 2's compute (the set's previous reader), and its
    compute waits for its own upload and for step i - 2's download (the set's
    previous output).  So step i + 1's upload and step i - 1's download overlap
    step i's kernels, and each step still moves all of its own bytes.

    make_plan: () -> a PrefillPlan / DecodePlan (anything with .stages and .out)
    host_inputs: name -> pinned host tensor, the shapes and dtypes of one step's inputs
    resident: name -> device tensor that every step reads in place (e.g. a KV cache)
    """

    def __init__(self, make_plan, host_inputs, resident=None, device="cuda"):
        dev = torch.device(device)
        self.plans = [make_plan(), make_plan()]
        self.inputs = []
        for _ in range(2):
            x = {k: torch.empty(v.shape, dtype=v.dtype, device=dev) for k, v in host_inputs.items()}
            x.update(resident or {})
            self.inputs.append(x)
        self.up, self.comp, self.down = (torch.cuda.Stream(device=dev) for _ in range(3))
        self.stages = [p.stages(x, self.comp) for p, x in zip(self.plans, self.inputs)]
        ev = lambda: [torch.cuda.Event(), torch.cuda.Event()]
        self.up_done, self.comp_done, self.down_done = ev(), ev(), ev()
        self.used = [False, False]

    def run(self, step_inputs, step_outputs, before_compute=None):
        """step_inputs[i]: name -> pinned host tensor; step_outputs[i]: pinned host
        tensor shaped like plan.out.  before_compute(i), if given, runs on the
        compute stream ahead of step i's kernels.  Returns without waiting;
        synchronize (or wait on self.down) before reading the outputs."""
        for i, (hin, hout) in enumerate(zip(step_inputs, step_outputs)):
            b = i % 2
            with torch.cuda.stream(self.up):
                if self.used[b]:
                    self.up.wait_event(self.comp_done[b])
                for k, t in hin.items():
                    self.inputs[b][k].copy_(t, non_blocking=True)
                self.up_done[b].record(self.up)
            with torch.cuda.stream(self.comp):
                self.comp.wait_event(self.up_done[b])
                if self.used[b]:
                    self.comp.wait_event(self.down_done[b])
                if before_compute is not None:
                    before_compute(i)
                for _, fn in self.stages[b]:
                    fn()
                self.comp_done[b].record(self.comp)
            with torch.cuda.stream(self.down):
                self.down.wait_event(self.comp_done[b])
                hout.copy_(self.plans[b].out, non_blocking=True)
                self.down_done[b].record(self.down)
            self.used[b] = True

    def dev_status(self) -> int:
        """OR of both plans' device status words (synchronizes)."""
        return int(self.plans[0].dev_status.item()) | int(self.plans[1].dev_status.item())
