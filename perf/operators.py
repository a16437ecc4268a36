"""Workloads of the cache operators: appending rotated keys and values to a
(paged) cache held in 16 or 8 bits, and selected-key attention over the 8-bit
cache.

``run`` makes one pass in plain torch, or, with ``own`` set, through the
library.  A row r = b * T + t of a step is token t of sequence b; n_valid[r] is
the number of cached tokens it sees (its own position + 1), 0 for padding.
"""

import math

import torch

own = False

PAGE = 64
E_MIN, E_MAX = -64, 64   # exponents of the cache scales
FP8_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    attn = dict(op="attn", paged=True, pad=False, sb=64, d=128)
    app = dict(op="append", paged=True, pad=False, sb=64, d=128, q8=True, rot=128, inter=False, kI8=False, D_I=64)
    return [
        # one user's next token: the smallest decode step
        dict(attn, name="attn_decode_1x4k", B=1, T=1, L0=4096, L1=4096, Hq=16, K=1024, W=128),
        # the long-context decode step over a contiguous cache
        dict(attn, name="attn_decode_8x128k", B=8, T=1, L0=131072, L1=131072, Hq=64, K=2048, W=512, paged=False),
        # the same over a shared pool of pages with uneven contexts
        dict(attn, name="attn_decode_paged_16x256k", B=16, T=1, L0=16384, L1=262144, Hq=64, K=2048, W=512),
        # several draft tokens a sequence are verified at once
        dict(attn, name="attn_verify_32x4", B=32, T=4, L0=1000, L1=30000, Hq=32, K=1024, W=128, sb=32),
        # a chunk of one prompt
        dict(attn, name="attn_chunk_1x2048", B=1, T=2048, L0=8192, L1=8192, Hq=16, K=1024, W=128, paged=False),
        # chunks of several prompts padded to one length, the largest attention step
        dict(attn, name="attn_chunk_4x1024_padded", B=4, T=1024, L0=20000, L1=65536, Hq=64, K=2048, W=512, pad=True),
        # short prompts of odd sizes, small heads
        dict(attn, name="attn_odd_3x37", B=3, T=37, L0=40, L1=300, Hq=5, d=64, K=64, W=32, sb=16, pad=True),
        # the append of one decode step, 8-bit cache
        dict(app, name="append_decode_16_q8", B=16, T=1, L0=100, L1=2000, Hq=64, kI8=True),
        # the append of one decode step, 16-bit cache
        dict(app, name="append_decode_64_bf16", B=64, T=1, L0=10, L1=500, Hq=16, q8=False),
        # a whole prompt enters the 8-bit cache: the largest append
        dict(app, name="append_prompt_8192_q8", B=1, T=8192, L0=8192, L1=8192, Hq=64, kI8=True),
        # uneven chunks that begin inside a block, partial interleaved rotation
        dict(app, name="append_ragged_7x333_q8", B=7, T=333, L0=340, L1=1500, Hq=5, d=64, sb=16, rot=32, inter=True,
             pad=True),
        # two prompts enter a contiguous 16-bit cache
        dict(app, name="append_prompt_2x2048_bf16", B=2, T=2048, L0=2048, L1=4100, Hq=16, q8=False, inter=True,
             paged=False, D_I=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 128])
    c = dict(op=rng.choice(["attn", "attn", "append"]), paged=rng.random() < 0.7, d=d, sb=rng.choice([1, 8, 16, 32, 64, 64]),
             Hq=rng.randint(1, 64))
    if c["op"] == "attn":
        B = _log(rng, 1, 64)
        c.update(B=B, T=_log(rng, 1, 2048 // B))
        c.update(K=_log(rng, 1, 2048), W=rng.choice([0, 1, 32, 100, 512]))
        L0 = _log(rng, max(c["T"], 16), 40000)
        c.update(L0=L0, L1=rng.randint(L0, 2 * L0))
    else:
        B = _log(rng, 1, 64)
        c.update(B=B, T=_log(rng, 1, 4096 // B))
        L0 = rng.randint(c["T"], c["T"] + 500)
        c.update(L0=L0, L1=L0 + rng.randint(0, 1000), q8=rng.random() < 0.6, rot=rng.choice([0, 32, 64, d]),
                 inter=rng.random() < 0.5, D_I=rng.choice([32, 64]), kI8=rng.random() < 0.5)
    c["pad"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- sizes of a case
def _lengths(c):
    """(cached tokens after the step, new tokens) of each sequence."""
    out = []
    for b in range(c["B"]):
        L = c["L0"] + int((c["L1"] - c["L0"]) * ((0.35 + 0.618034 * b) % 1.0))
        n = max(1, int(c["T"] * ((0.9 + 0.37 * b) % 1.0))) if c["pad"] else c["T"]
        out.append((L, min(n, L)))
    return out


def _n_keys(c, n):
    """Keys that the row which sees n cached tokens attends to, when its top-K is spread evenly over them: the window,
    and the selected positions in front of it."""
    if n <= c["K"]:
        return n
    front = max(0, n - c["W"])
    return min(n - front + (front * c["K"] + n - 1) // n, n)


def work(c):
    d, Hq, lens = c["d"], c["Hq"], _lengths(c)
    rows = sum(n for _, n in lens)
    if c["op"] == "attn":
        keys = cached = 0
        for L, n in lens:
            step = max(1, n // 64)
            sampled = [_n_keys(c, L - n + t + 1) for t in range(0, n, step)]
            mine = sum(sampled) * n // len(sampled)
            keys += mine
            cached += min(mine, L)
        return {"bytes": rows * (4.0 * Hq * d + 4 * Hq + 4 * c["K"]) + cached * (2.0 * d + 8.0 / c["sb"]),
                "flops": 4.0 * Hq * d * keys}
    size = 1 if c["q8"] else 2
    per_row = 4.0 * Hq * d + 2 * d * (2 + size) + c["D_I"] * (2 + (1 if c["kI8"] else 2))
    return {"bytes": rows * per_row + (8.0 * rows / c["sb"] if c["q8"] else 0.0), "flops": 3.0 * rows * (Hq + 1) * c["rot"]}


# ---------------------------------------------------------------- inputs
def _pow2_scale(amax):
    """The smallest power of two s (within the range of the cache scales) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(E_MIN, E_MAX)
    return torch.ldexp(torch.ones_like(amax), e.where(amax > 0, torch.full_like(e, E_MIN)))


def _filled(rows, c, gen, dev):
    """A cache side in 8 bits: uneven tokens and a few strong channels, as projections give."""
    x = torch.randn(rows, c["d"], generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=dev))
    x[:, ::17] *= 3.0
    blocks = x.view(-1, c["sb"], c["d"])
    s = _pow2_scale(blocks.abs().amax((1, 2)))
    codes = (blocks / s[:, None, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(rows, c["d"]).contiguous(), s.contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    B, T, d, Hq = c["B"], c["T"], c["d"], c["Hq"]
    lens = _lengths(c)
    nv = torch.zeros(B, T, dtype=torch.int32)
    for b, (L, n) in enumerate(lens):
        nv[b, :n] = torch.arange(L - n + 1, L + 1, dtype=torch.int32)
    nv = nv.view(-1)
    rows_host = nv.nonzero().view(-1)
    pages = [-(-L // PAGE) for L, _ in lens]
    max_pages = max(pages)
    st = dict(c=c, nv=nv.to(dev), rows=rows_host.to(dev), max_pages=max_pages, S_max=max_pages * PAGE, pt=None, pool_pages=0)
    if c["paged"]:
        total = sum(pages) + 3
        order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
        pt, at = torch.zeros(B, max_pages, dtype=torch.int32, device=dev), 0
        for b, n in enumerate(pages):
            pt[b, :n] = order[at:at + n]
            at += n
        st.update(pt=pt, pool_pages=total)
        n_rows = total * PAGE
    else:
        n_rows = B * st["S_max"]
    bf = lambda *s: torch.randn(*s, generator=gen, device=dev).bfloat16()  # noqa: E731
    st["q"] = bf(B * T, Hq, d)
    if c["op"] == "attn":
        st["kc"], st["ks"] = _filled(n_rows, c, gen, dev)
        st["vc"], st["vs"] = _filled(n_rows, c, gen, dev)
        K, n = c["K"], st["nv"].long()[:, None]
        i = torch.arange(K, device=dev)[None]
        lo, hi = i * n // K, (i + 1) * n // K   # one position out of each of K strata: ascending, none twice
        u = torch.rand(B * T, K, generator=gen, device=dev, dtype=torch.float64)
        pick = lo + torch.minimum((u * (hi - lo)).long(), (hi - lo - 1).clamp(min=0))
        st["topk"] = torch.where(n > K, pick, torch.where(i < n, i, -1)).to(torch.int32).contiguous()
        st["out"] = torch.empty(B * T, Hq, d, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty(B * T, Hq, dtype=torch.float32, device=dev)
    else:
        st["k"], st["v"] = bf(B * T, d) * 2, bf(B * T, d)
        st["kI"] = torch.randint(-3, 4, (B * T, c["D_I"]), generator=gen, device=dev).bfloat16()
        half = torch.arange(max(c["rot"] // 2, 1), device=dev, dtype=torch.float64)
        st["inv_freq"] = (10000.0 ** (-half / max(c["rot"] // 2, 1))).float()
        if c["q8"]:
            st["kc"], st["ks"] = _filled(n_rows, c, gen, dev)
            st["vc"], st["vs"] = _filled(n_rows, c, gen, dev)
        else:
            st["kc"], st["vc"] = bf(n_rows, d), bf(n_rows, d)
        st["kIc"] = torch.randint(-3, 4, (n_rows, c["D_I"]), generator=gen, device=dev).bfloat16()
        if c["kI8"]:
            st["kIc"] = st["kIc"].to(torch.float8_e4m3fn).view(torch.uint8)
        st["q_out"] = torch.zeros_like(st["q"])
    st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return st


# ---------------------------------------------------------------- plain form
def _slots(st, b, pos):
    """Cache rows of positions `pos` of sequences `b` (long tensors of one shape)."""
    if st["pt"] is None:
        return b * st["S_max"] + pos
    return st["pt"][b, pos // PAGE].long() * PAGE + pos % PAGE


def _plain_attn(st):
    c, nv = st["c"], st["nv"].long()
    R, W = nv.numel(), c["W"]
    b = torch.arange(R, device=nv.device)[:, None] // c["T"]
    p = nv[:, None] - 1
    top = st["topk"].long()
    win = p - W + 1 + torch.arange(W, device=nv.device)[None]
    pos = torch.cat([top, win], 1)
    ok = torch.cat([(top >= 0) & (top <= p - W), (win >= 0) & (p >= 0)], 1)
    slot = _slots(st, b.expand_as(pos), pos.clamp(min=0))
    blk = slot // c["sb"]
    k = st["kc"].view(torch.float8_e4m3fn)[slot].float() * st["ks"][blk][..., None]
    x = torch.einsum("rhd,rsd->rhs", st["q"].float(), k) / math.sqrt(c["d"])
    del k
    x = x.masked_fill(~ok[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(x - m)
    l = e.sum(-1)
    v = st["vc"].view(torch.float8_e4m3fn)[slot].float() * st["vs"][blk][..., None]
    o = torch.einsum("rhs,rsd->rhd", e, v) / l.clamp(min=1e-30)[..., None]
    return o.bfloat16(), m[..., 0] + torch.log(l)


def _plain_rot(x, cos, sin, c):
    """x [n, heads, d] fp32, cos / sin [n, rot / 2]."""
    rot = c["rot"]
    if rot == 0:
        return x
    y, cos, sin = x.clone(), cos[:, None], sin[:, None]
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_q8(st, x, codes, scales, pos, slot, first):
    """Quantise the new rows x [n, d] into their blocks; `first`: rows that are the first new token of a sequence."""
    sb, n_blk = st["c"]["sb"], scales.numel()
    blk = slot // sb
    amax = torch.zeros(n_blk, device=x.device).scatter_reduce(0, blk, x.abs().amax(-1), "amax")
    fresh = torch.zeros(n_blk, dtype=torch.bool, device=x.device)
    fresh[blk] = True
    fresh_start = torch.zeros(n_blk, device=x.device).scatter_reduce(0, blk, (pos % sb == 0).float(), "amax") > 0
    old = scales.clone()
    need = _pow2_scale(amax)
    new = torch.where(fresh, torch.where(fresh_start, need, torch.maximum(need, old)), old)
    # earlier tokens of the block that a sequence's first new token falls into
    fb, off = blk[first], pos[first] % sb
    view = codes.view(torch.float8_e4m3fn).view(n_blk, sb, -1)
    kept = (view[fb].float() * (old[fb] / new[fb])[:, None, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    earlier = (torch.arange(sb, device=x.device)[None] < off[:, None])[..., None]
    bytes_ = codes.view(n_blk, sb, -1)
    bytes_[fb] = torch.where(earlier, kept.view(torch.uint8), bytes_[fb])
    scales.copy_(new)
    codes[slot] = (x / new[blk][:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(st):
    c, rows = st["c"], st["rows"]
    pos = st["nv"][rows].long() - 1
    b = rows // c["T"]
    slot = _slots(st, b, pos)
    a = pos[:, None].double() * st["inv_freq"].double()[None]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    st["q_out"][rows] = _plain_rot(st["q"][rows].float(), cos, sin, c).bfloat16()
    k = _plain_rot(st["k"][rows].float()[:, None], cos, sin, c)[:, 0]
    if c["q8"]:
        first = torch.arange(c["B"], device=rows.device) * c["T"]       # every sequence has a new token
        at = torch.searchsorted(rows, first)
        _plain_q8(st, k, st["kc"], st["ks"], pos, slot, at)
        _plain_q8(st, st["v"][rows].float(), st["vc"], st["vs"], pos, slot, at)
    else:
        st["kc"][slot] = k.bfloat16()
        st["vc"][slot] = st["v"][rows]
    kI = st["kI"][rows]
    st["kIc"][slot] = kI.float().clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8) if c["kI8"] else kI


# ---------------------------------------------------------------- one pass
def _append_outputs(st):
    f8 = lambda t: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t  # noqa: E731
    out = dict(q=st["q_out"], k=f8(st["kc"]), v=f8(st["vc"]), kI=f8(st["kIc"]))
    if st["c"]["q8"]:
        out.update(k_scale=st["ks"], v_scale=st["vs"])
    return out


def run(st):
    c = st["c"]
    if not own:
        if c["op"] == "attn":
            return _plain_attn(st)
        _plain_append(st)
        return _append_outputs(st)
    import fine_grained_top_b200 as sa
    B, T, d, Hq = c["B"], c["T"], c["d"], c["Hq"]
    where = (st["pt"], st["max_pages"], st["pool_pages"], PAGE, st["S_max"])
    if c["op"] == "attn":
        sa.sa_sparse_attn_q8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], c["sb"], *where, st["nv"], st["topk"], c["K"],
                             c["W"], B, T, Hq, d, 1.0 / math.sqrt(d), st["out"], st["lse"], st["status"])
        return st["out"], st["lse"]
    rows = (st["q"], Hq * d, st["q_out"], st["k"], d, st["v"], d, st["kI"], c["D_I"], st["nv"], *where, B, T, Hq, d, c["D_I"],
            st["inv_freq"], c["rot"], int(c["inter"]))
    if c["q8"]:
        sa.sa_cache_append_q8(*rows, st["kc"], st["vc"], st["ks"], st["vs"], c["sb"], st["kIc"], int(c["kI8"]), st["status"])
    else:
        sa.sa_cache_append(*rows, st["kc"], st["vc"], st["kIc"], int(c["kI8"]), st["status"])
    return _append_outputs(st)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_attn(st):
    """Row by row groups: the selected set, its scores and their softmax, all in 64 bits."""
    c, R = st["c"], st["nv"].numel()
    f8 = lambda t, s: t.view(torch.float8_e4m3fn).double() * s.double()[..., None]  # noqa: E731
    out = torch.zeros(R, c["Hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((R, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    nv = st["nv"].tolist()
    group = max(1, 400000 // (c["K"] + c["W"] + 1))
    for r0 in range(0, R, group):
        r1 = min(R, r0 + group)
        n = st["nv"][r0:r1].long()
        if max(nv[r0:r1]) == 0:
            continue
        seq = torch.arange(r0, r1, device="cuda") // c["T"]
        before = (n - c["W"]).clamp(min=0)   # positions in front of the window
        top = st["topk"][r0:r1].long()
        tail = before[:, None] + torch.arange(c["W"], device="cuda")
        member = torch.cat([(top >= 0) & (top < before[:, None]), tail < n[:, None]], 1)
        at = torch.cat([top, tail], 1).masked_fill(~member, 0)
        slot = _slots(st, seq[:, None].expand_as(at), at)
        s = torch.matmul(st["q"][r0:r1].double(), f8(st["kc"][slot], st["ks"][slot // c["sb"]]).transpose(1, 2))
        s = torch.where(member[:, None], s * c["d"] ** -0.5, -math.inf)
        z = torch.logsumexp(s, -1)
        some = member.any(1)
        w = torch.where(some[:, None, None], torch.exp(s - torch.where(some[:, None], z, 0.0)[..., None]), 0.0)
        out[r0:r1] = torch.matmul(w, f8(st["vc"][slot], st["vs"][slot // c["sb"]]))
        lse[r0:r1] = z
    return out, lse


def _exact_append(st):
    """Token by token of each sequence on the host, in 64 bits; 8-bit caches as unrounded multiples of their scales."""
    c = st["c"]
    sb, rot, nv = c["sb"], c["rot"], st["nv"].cpu().view(c["B"], c["T"]).long()
    host = lambda t: t.cpu().double()  # noqa: E731
    code = lambda t: host(t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t)  # noqa: E731
    q, k, v, kI = (host(st[n]).view(c["B"], c["T"], -1, w) for n, w in
                   (("q", c["d"]), ("k", c["d"]), ("v", c["d"]), ("kI", c["D_I"])))
    pt = None if st["pt"] is None else st["pt"].cpu().long()
    q_out, kc, vc, kIc = host(st["q_out"]).view(c["B"], c["T"], -1, c["d"]), code(st["kc"]), code(st["vc"]), code(st["kIc"])
    scales = [host(st["ks"]), host(st["vs"])] if c["q8"] else []
    first = torch.arange(0, rot, 2) if c["inter"] else torch.arange(rot // 2)
    second = first + (1 if c["inter"] else rot // 2)

    def turned(x, angle):
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    for b in range(c["B"]):
        n = int((nv[b] > 0).sum())
        p = nv[b, :n] - 1
        slot = b * st["S_max"] + p if pt is None else pt[b, p // PAGE] * PAGE + p % PAGE
        angle = p[:, None].double() * host(st["inv_freq"])[: rot // 2]
        q_out[b, :n] = turned(q[b, :n], angle)
        new = [turned(k[b, :n], angle)[:, 0], v[b, :n, 0]]
        kIc[slot] = kI[b, :n, 0]
        if not c["q8"]:
            kc[slot], vc[slot] = new
            continue
        for x, cache, scale in zip(new, (kc, vc), scales):
            for g in torch.unique(p // sb).tolist():
                mine = (p // sb == g).nonzero()[:, 0]
                rows = slot[mine]
                blk = int(rows[0]) // sb
                top = float(x[mine].abs().max())
                e = max(E_MIN, math.ceil(math.log2(top / FP8_MAX))) if top > 0 else E_MIN
                s = 2.0 ** min(e, E_MAX)
                earlier = int(p[mine[0]]) % sb
                if earlier:
                    s = max(s, float(scale[blk]))
                    cache[blk * sb: blk * sb + earlier] *= float(scale[blk]) / s
                scale[blk] = s
                cache[rows] = x[mine] / s
    out = dict(q=q_out.reshape(-1, c["Hq"], c["d"]), k=kc, v=vc, kI=kIc)
    if c["q8"]:
        out.update(k_scale=scales[0], v_scale=scales[1])
    return out


def exact(c, seed):
    st = prepare(c, seed)
    return _exact_attn(st) if c["op"] == "attn" else _exact_append(st)
