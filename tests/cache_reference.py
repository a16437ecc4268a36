"""Plain 64-bit forms of the cache append and of the attention over an 8-bit
cache, on the CPU, with the tolerances that the number formats allow.

Tolerances: bf16 rounding is off by at most 2^-8 of the value, e4m3 by 2^-4 of
it (2^-10 of the scale among the subnormals), fp32 by 2^-24."""

import math

import torch

E4M3 = torch.float8_e4m3fn


def rows_of(lens, news, T, left=False):
    """n_valid [B*T] of sequences that hold lens[b] tokens after the step, the last news[b] of them new."""
    nv = torch.zeros(len(lens), T, dtype=torch.int32)
    for b, (L, n) in enumerate(zip(lens, news)):
        at = T - n if left else 0
        nv[b, at:at + n] = torch.arange(L - n + 1, L + 1, dtype=torch.int32)
    return nv.view(-1)


def paged_table(lens, gen, spare=2):
    """(page_table [B, max_pages], pool_pages): every sequence's pages drawn from one shuffled pool."""
    pages = [max(1, -(-L // 64)) for L in lens]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=gen).to(torch.int32)
    pt, at = torch.zeros(len(lens), max(pages), dtype=torch.int32), 0
    for b, n in enumerate(pages):
        pt[b, :n] = order[at:at + n]
        at += n
    return pt, total


def slot_of(pt, S_max, b, p):
    return b * S_max + p if pt is None else int(pt[b, p // 64]) * 64 + p % 64


def rotate(x, p, inv_freq, rot, inter):
    """x [..., d] float64 rotated to position p, and a bound of fp32 evaluation errors."""
    first = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    second = first + (1 if inter else rot // 2)
    a = p * inv_freq[:rot // 2].double()
    y, slack = x.clone(), torch.zeros_like(x)
    u, v = x[..., first], x[..., second]
    y[..., first] = u * torch.cos(a) - v * torch.sin(a)
    y[..., second] = v * torch.cos(a) + u * torch.sin(a)
    # the angle in fp32 half turns (pi 2^-25), sine and cosine within 2 ulp (2^-23),
    # two products and a sum (3 * 2^-24): together under 2^-21 of |u| + |v|
    slack[..., first] = slack[..., second] = (u.abs() + v.abs()) * 2.0 ** -21
    return y, slack


def scale_for(amax):
    if amax <= 0:
        return 2.0 ** -64
    m, e = math.frexp(amax)
    return 2.0 ** min(64, max(-64, e - 9 if m <= 0.875 else e - 8))


def to_e4m3(x):
    """Codes of float64 values (exact in fp32 here, or far from a border)."""
    return x.clamp(-448, 448).to(torch.float32).to(E4M3).view(torch.uint8)


def of_e4m3(codes):
    return codes.view(E4M3).to(torch.float64)


def finite_max(x):
    x = x.abs()
    return float(torch.where(torch.isfinite(x), x, torch.zeros_like(x)).max())


def append_block_q8(codes, scale, blk, sb, first_off, x):
    """New values x [n, d] (float64) enter tokens first_off.. of block blk: codes [rows, d] uint8 and scale [blocks]
    (float64) are updated in place.  Returns the new codes' exact values / scale."""
    need = scale_for(finite_max(x))
    r0 = blk * sb
    if first_off > 0:
        old = min(max(float(scale[blk]), 2.0 ** -64), 2.0 ** 64) if not math.isnan(float(scale[blk])) else 2.0 ** -64
        new = max(need, old)
        if new != old:
            codes[r0:r0 + first_off] = to_e4m3(of_e4m3(codes[r0:r0 + first_off]) * (old / new))
    else:
        new = need
    scale[blk] = new
    y = x / new
    codes[r0 + first_off:r0 + first_off + len(x)] = to_e4m3(y)
    return y


def attention(q, kc, vc, ks, vs, sb, pt, S_max, nv, topk, W, T, scale):
    """(out, lse, tolerance of out, tolerance of lse), float64, and the set sizes; caches as [rows, d] codes."""
    R, Hq, d = q.shape
    out, lse = torch.zeros(R, Hq, d, dtype=torch.float64), torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    sizes = []
    for r in range(R):
        p = int(nv[r]) - 1
        top = [e for e in topk[r].tolist() if 0 <= e <= p - W] if topk is not None else []
        keys = top + list(range(max(0, p - W + 1), p + 1))
        sizes.append(len(keys))
        if not keys:
            continue
        slots = torch.tensor([slot_of(pt, S_max, r // T, s) for s in keys])
        cl = lambda s: s.double().clamp(2.0 ** -64, 2.0 ** 64)  # noqa: E731
        kcode, vcode = of_e4m3(kc[slots]), of_e4m3(vc[slots])
        kscale, vscale = cl(ks[slots // sb]), cl(vs[slots // sb])
        qr = q[r].double()
        x = (qr @ kcode.T) * kscale * scale
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - z[:, None])
        wv = w * vscale
        out[r], lse[r] = wv @ vcode, z
        # q is split into two e4m3 parts of a row-wide scale: exact down to 2^-10 of
        # the row's largest value, below it off by 2^-10 / 224 of that value
        dx = (qr.abs().max() * 2.0 ** -10 / 224 * kcode.abs().sum(-1) * kscale * abs(scale)).max()
        # fp32 scores: 2^-22 of their products' magnitudes; exp2 2^-22; sums of n terms n 2^-24
        mag = ((qr.abs() @ kcode.abs().T) * kscale * abs(scale)).max()
        rel = float(dx + mag * 2.0 ** -22) * 2 + 2.0 ** -18 + len(keys) * 2.0 ** -24
        # P in fp16 (2^-12 of its value) and two e4m3 parts, the second times 16: 2^-8 of
        # its value (half a step of the rest), and 2^-14 among the second part's
        # subnormals, where the largest P is at least 2
        aw = wv @ vcode.abs()
        floor = wv.max(-1).values[:, None] * vcode.abs().sum(0)[None] * 2.0 ** -15
        tol_o[r] = 2.0 ** -8 * out[r].abs() + (2.0 ** -8 + 2.0 ** -12 + rel) * aw + floor
        tol_l[r] = rel + 2.0 ** -22 * z.abs()
    return out, lse, tol_o, tol_l, sizes
