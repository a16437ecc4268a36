"""GPU tests of the cache append (16 and 8 bits) and of the attention over the
8-bit cache against plain 64-bit forms, alone and run together."""

import math

import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    import fine_grained_top_b200 as m
    return m


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- append
def append_inputs(lens, news, T, Hq, d, D_I, rot, inter, q8, sb, kI8, paged, seed, left=False, S_max=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    x = dict(nv=ref.rows_of(lens, news, T, left), inv=(10000.0 ** (-torch.arange(max(rot // 2, 1)).double() / max(rot // 2, 1))).float())
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    x.update(q=bf(B * T, Hq, d), k=bf(B * T, d) * 3, v=bf(B * T, d), kI=bf(B * T, D_I) * 4)
    x["S_max"] = S_max or max(64, -(-max(lens) // 64) * 64)
    x["pt"], x["pool"] = ref.paged_table(lens, g) if paged else (None, 0)
    n = x["pool"] * 64 if paged else B * x["S_max"]
    if q8:
        for s in "kv":
            codes = torch.randint(0, 256, (n, d), generator=g, dtype=torch.uint8)
            codes[(codes & 127) == 127] = 0   # no NaN among the old codes
            x[s + "c"] = codes
            x[s + "s"] = torch.exp2(torch.randint(-9, -3, (n // sb,), generator=g).float())
    else:
        x["kc"], x["vc"] = bf(n, d), bf(n, d)
    x["kIc"] = torch.randint(0, 120, (n, D_I), generator=g, dtype=torch.uint8) if kI8 else bf(n, D_I)
    return x


def run_append(sa, x, T, Hq, d, D_I, rot, inter, q8, sb, kI8, dev_x=None):
    """The call on copies on the GPU; returns the device tensors (q_out, kc, vc, kIc, ks, vs) and the status word."""
    B = x["nv"].numel() // T
    y = dev_x or {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    y["q_out"] = torch.full_like(y["q"], 7.0)
    y["status"] = status_word()
    pt = y.get("pt")
    args = (y["q"], Hq * d, y["q_out"], y["k"], d, y["v"], d, y["kI"], D_I, y["nv"], pt, pt.shape[1] if pt is not None else 0,
            x["pool"], 64, x["S_max"], B, T, Hq, d, D_I, y["inv"], rot, int(inter))
    if q8:
        sa.sa_cache_append_q8(*args, y["kc"], y["vc"], y["ks"], y["vs"], sb, y["kIc"], int(kI8), y["status"])
    else:
        sa.sa_cache_append(*args, y["kc"], y["vc"], y["kIc"], int(kI8), y["status"])
    torch.cuda.synchronize()
    return y


def check_append(x, y, T, Hq, d, D_I, rot, inter, q8, sb, kI8):
    nv, B = x["nv"].view(-1, T), x["nv"].numel() // T
    got = {n: y[n].cpu() for n in ("q_out", "kc", "vc", "kIc") + (("ks", "vs") if q8 else ())}
    want_kI, written = x["kIc"].clone(), torch.zeros(len(x["kc"]), dtype=torch.bool)
    want = {n: x[n].clone() for n in ("kc", "vc")}
    scales = {n: x[n].double().clone() for n in ("ks", "vs")} if q8 else {}
    for b in range(B):
        rows = [t for t in range(T) if nv[b, t] > 0]
        ks, slots, pos = [], [], []
        for t in range(T):
            r = b * T + t
            if nv[b, t] == 0:   # padding: untouched
                assert (got["q_out"][r] == 7.0).all()
                continue
            p = int(nv[b, t]) - 1
            yq, sq = ref.rotate(x["q"][r].double(), p, x["inv"], rot, inter)
            err = (got["q_out"][r].double() - yq).abs()
            assert (err <= 2.0 ** -8 * yq.abs() + sq).all(), ("q", b, t, float((err - 2.0 ** -8 * yq.abs() - sq).max()))
            s = ref.slot_of(x["pt"], x["S_max"], b, p)
            written[s] = True
            slots.append(s)
            pos.append(p)
            ks.append(ref.rotate(x["k"][r].double(), p, x["inv"], rot, inter))
            want_kI[s] = ref.to_e4m3(x["kI"][r].double()) if kI8 else x["kI"][r]
        if not rows:
            continue
        yk, sk = torch.stack([k for k, _ in ks]), torch.stack([s for _, s in ks])
        slot_t = torch.tensor(slots)
        xv = x["v"][[b * T + t for t in rows]]
        if not q8:
            err = (got["kc"][slot_t].double() - yk).abs()
            assert (err <= 2.0 ** -8 * yk.abs() + sk).all()
            want["vc"][slot_t] = xv
            continue
        for i0 in range(len(slots)):   # the new tokens of one block at a time
            if i0 and pos[i0] % sb:
                continue
            n = 1
            while i0 + n < len(slots) and pos[i0 + n] % sb:
                n += 1
            blk, off = slots[i0] // sb, pos[i0] % sb
            ref.append_block_q8(want["vc"], scales["vs"], blk, sb, off, xv[i0:i0 + n].double())
            ref.append_block_q8(want["kc"], scales["ks"], blk, sb, off, yk[i0:i0 + n])
            s = float(scales["ks"][blk])
            val = ref.of_e4m3(got["kc"][slot_t[i0:i0 + n]]) * s
            lim = 2.0 ** -4 * yk[i0:i0 + n].abs() + 2.0 ** -10 * s + sk[i0:i0 + n]
            assert ((val - yk[i0:i0 + n]).abs() <= lim).all()
    if q8:
        assert torch.equal(got["ks"].double(), scales["ks"]) and torch.equal(got["vs"].double(), scales["vs"])
        assert torch.equal(got["vc"], want["vc"])                       # new values, earlier tokens and the rest, bit for bit
        assert torch.equal(got["kc"][~written], want["kc"][~written])   # rescaled earlier keys, untouched rest
    else:
        assert torch.equal(got["vc"], want["vc"])
        assert torch.equal(got["kc"][~written], x["kc"][~written])
    assert torch.equal(got["kIc"].view(torch.uint8), want_kI.view(torch.uint8))
    assert int(y["status"].item()) == 0


APPENDS = [
    # lens, news, T, Hq, d, D_I, rot, inter, sb, kI8, paged
    ([1], [1], 1, 1, 64, 32, 64, False, 64, False, True),
    ([1, 64, 65, 130], [1, 1, 1, 1], 1, 16, 128, 64, 128, False, 64, True, True),
    ([17, 200], [1, 1], 1, 64, 128, 128, 64, True, 16, True, False),
    ([100, 7, 63], [100, 7, 63], 100, 5, 128, 64, 128, False, 64, False, True),
    ([150, 90, 300], [93, 0, 81], 93, 3, 128, 64, 32, True, 32, True, True),
    ([65, 129], [2, 66], 66, 7, 64, 32, 16, False, 1, True, False),
    ([500], [197], 197, 64, 64, 64, 0, False, 8, False, True),
    ([191, 64], [128, 64], 128, 2, 128, 32, 96, False, 64, False, True),
    ([40, 41, 42], [13, 14, 15], 15, 33, 64, 128, 48, True, 2, True, True),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("q8", [False, True])
def test_append(sa, case, q8):
    lens, news, T, Hq, d, D_I, rot, inter, sb, kI8, paged = APPENDS[case]
    x = append_inputs(lens, news, T, Hq, d, D_I, rot, inter, q8, sb, kI8, paged, seed=case, left=case % 2 == 1)
    y = run_append(sa, x, T, Hq, d, D_I, rot, inter, q8, sb, kI8)
    check_append(x, y, T, Hq, d, D_I, rot, inter, q8, sb, kI8)


def test_append_q8_longest_call(sa):
    """131072 rows in one call, padded in front: every block's scale and codes."""
    T, n, d, sb = 131072, 130_990, 64, 64
    g = torch.Generator().manual_seed(13)
    k = torch.randn(T, d, generator=g).mul(torch.exp2(torch.randint(-9, 9, (T, 1), generator=g).float())).bfloat16()
    nv = ref.rows_of([n], [n], T, left=True).cuda()
    kc, vc = (torch.full((T, d), 0x11, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((T // sb,), 9.0, device="cuda") for _ in range(2))
    st, kd, vd = status_word(), k.cuda(), k.flip(1).contiguous().cuda()
    sa.sa_cache_append_q8(None, 0, None, kd, d, vd, d, None, 0, nv, None, 0, 0, 64, T, 1, T, 0, d, 0, None, 0, 0, kc, vc, ks, vs,
                          sb, None, 0, st)
    assert int(st.item()) == 0
    x = torch.zeros(T, d, dtype=torch.float64)
    x[:n] = k[T - n:].double()
    amax = x.view(-1, sb * d).abs().max(1).values
    used = -(-n // sb)
    scale = torch.tensor([ref.scale_for(float(a)) for a in amax[:used]], dtype=torch.float64)
    assert torch.equal(ks.cpu().double()[:used], scale) and torch.equal(vs.cpu().double()[:used], scale)
    assert (ks.cpu()[used:] == 9.0).all()
    want = ref.to_e4m3(x[:n] / scale.repeat_interleave(sb)[:n, None])
    assert torch.equal(kc.cpu()[:n], want) and torch.equal(vc.cpu()[:n], want.flip(1))
    assert (kc.cpu()[n:] == 0x11).all() and (vc.cpu()[n:] == 0x11).all()


def test_append_far_positions(sa):
    """Positions up to 2^31 - 64: the angle keeps its accuracy (the page table is short by page 0 of the pool alone)."""
    T, Hq, d, D_I = 3, 2, 128, 64
    for last in (524288, 20_000_011):
        g = torch.Generator().manual_seed(last)
        x = append_inputs([70], [3], T, Hq, d, D_I, 128, False, True, 64, False, True, seed=1)
        L = last
        x["nv"] = ref.rows_of([L], [3], T)
        n_pages = -(-L // 64)
        x["pt"] = torch.randint(0, x["pool"], (1, n_pages), generator=g, dtype=torch.int32)
        x["pt"][0, (L - 3) // 64], x["pt"][0, (L - 1) // 64] = 0, 1   # the pages that are written
        if (L - 3) // 64 == (L - 1) // 64:
            x["pt"][0, (L - 1) // 64] = 0
        y = run_append(sa, x, T, Hq, d, D_I, 128, False, True, 64, False)
        check_append(x, y, T, Hq, d, D_I, 128, False, True, 64, False)


@pytest.mark.parametrize("q8", [False, True])
def test_append_takes_slices_of_one_projection(sa, q8):
    T, Hq, d, D_I, rot = 9, 4, 128, 64, 128
    x = append_inputs([40, 9], [9, 9], T, Hq, d, D_I, rot, False, q8, 64, False, True, seed=5)
    whole = run_append(sa, x, T, Hq, d, D_I, rot, False, q8, 64, False)
    y = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    wide = torch.zeros(18, Hq * d + 2 * d + D_I + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :Hq * d] = y["q"].view(18, -1)
    wide[:, Hq * d:Hq * d + d], wide[:, Hq * d + d:Hq * d + 2 * d] = y["k"], y["v"]
    wide[:, Hq * d + 2 * d:-8] = y["kI"]
    ld, st = wide.shape[1], status_word()
    q_out = torch.empty_like(y["q"])
    args = (wide[:, :Hq * d], ld, q_out, wide[:, Hq * d:Hq * d + d], ld, wide[:, Hq * d + d:Hq * d + 2 * d], ld,
            wide[:, Hq * d + 2 * d:-8], ld, y["nv"], y["pt"], y["pt"].shape[1], x["pool"], 64, x["S_max"], 2, T, Hq, d, D_I,
            y["inv"], rot, 0)
    if q8:
        sa.sa_cache_append_q8(*args, y["kc"], y["vc"], y["ks"], y["vs"], 64, y["kIc"], 0, st)
    else:
        sa.sa_cache_append(*args, y["kc"], y["vc"], y["kIc"], 0, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(q_out, whole["q_out"])
    for n in ("kc", "vc", "kIc"):
        assert torch.equal(y[n], whole[n]), n


@pytest.mark.parametrize("q8", [False, True])
def test_append_without_queries_or_index_keys_and_in_place(sa, q8):
    T, Hq, d, D_I, rot = 5, 4, 64, 64, 64
    x = append_inputs([40, 9], [5, 5], T, Hq, d, D_I, rot, True, q8, 16, False, False, seed=6)
    whole = run_append(sa, x, T, Hq, d, D_I, rot, True, q8, 16, False)
    y = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    st, kI0 = status_word(), y["kIc"].clone()
    tail = (y["nv"], None, 0, 0, 64, x["S_max"], 2, T)
    cache = (y["kc"], y["vc"]) + ((y["ks"], y["vs"], 16) if q8 else ())
    f = sa.sa_cache_append_q8 if q8 else sa.sa_cache_append
    f(None, 0, None, y["k"], d, y["v"], d, None, 0, *tail, 0, d, 0, y["inv"], rot, 1, *cache, None, 0, st)
    torch.cuda.synchronize()
    assert torch.equal(y["kc"], whole["kc"]) and torch.equal(y["vc"], whole["vc"]) and torch.equal(y["kIc"], kI0)
    # q rotated in place; the appended tokens are the same again, so nothing else changes
    f(y["q"], Hq * d, y["q"], y["k"], d, y["v"], d, y["kI"], D_I, *tail, Hq, d, D_I, y["inv"], rot, 1, *cache, y["kIc"], 0, st)
    torch.cuda.synchronize()
    for n, m in (("q", "q_out"), ("kc", "kc"), ("vc", "vc"), ("kIc", "kIc")):
        assert torch.equal(y[n], whole[m]), n
    assert int(st.item()) == 0


def test_append_q8_special_values(sa):
    """Zeros, infinities and NaN among the new values: the scale goes by the finite ones."""
    T, Hq, d, D_I = 4, 1, 128, 32
    x = append_inputs([4, 68], [4, 4], T, Hq, d, D_I, 0, False, True, 64, False, False, seed=7)
    x["v"][:4] = 0
    x["v"][5, 3], x["v"][6, 4], x["v"][7, 5] = math.inf, -math.inf, math.nan
    x["k"][0, :] = 1e-30
    x["k"][1:4, :] = 0
    x["k"][4, 0] = 3.0e38   # beyond 448 * 2^64: saturates
    y = run_append(sa, x, T, Hq, d, D_I, 0, False, True, 64, False)
    vs, vc = y["vs"].cpu().view(2, -1), y["vc"].cpu().view(2, -1, d)
    assert vs[0, 0] == 2.0 ** -64 and (vc[0, :4] == 0).all()
    fin = torch.where(torch.isfinite(x["v"][4:]), x["v"][4:].double(), torch.zeros(()).double())
    assert vs[1, 1] == ref.scale_for(float(fin.abs().max()))
    codes = vc[1, 64:68].view(ref.E4M3).float()
    assert codes[1, 3] == 448 and codes[2, 4] == -448 and math.isnan(float(codes[3, 5])) and int(torch.isnan(codes).sum()) == 1
    ks = y["ks"].cpu().view(2, -1)
    assert ks[0, 0] == 2.0 ** -64 and ks[1, 1] == 2.0 ** 64
    assert y["kc"].cpu().view(2, -1, d)[1, 64, 0].view(ref.E4M3).float() == 448


def test_append_q8_token_by_token_grows_the_scale(sa):
    """64 single-token appends whose values grow: after each one the block equals the reference of the same steps."""
    d, sb = 64, 32
    x = append_inputs([64], [64], 64, 1, d, 32, 0, False, True, sb, False, True, seed=8)
    x["k"] *= torch.exp2(torch.arange(64) / 4.0)[:, None].bfloat16()
    y = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    codes, scale = x["kc"].clone(), x["ks"].double().clone()
    for t in range(64):
        s = ref.slot_of(x["pt"], 0, 0, t)
        ref.append_block_q8(codes, scale, s // sb, sb, t % sb, x["k"][t:t + 1].double())
        nv = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        sa.sa_cache_append_q8(None, 0, None, y["k"][t], d, y["v"][t], d, None, 0, nv, y["pt"], y["pt"].shape[1], x["pool"], 64, 0, 1,
                              1, 0, d, 0, None, 0, 0, y["kc"], y["vc"], y["ks"], y["vs"], sb, None, 0, None)
    assert torch.equal(y["kc"].cpu(), codes) and torch.equal(y["ks"].cpu().double(), scale)


def test_append_reports_bad_rows_and_leaves_the_caches(sa):
    T, Hq, d, D_I = 4, 2, 128, 64
    for q8 in (False, True):
        for what, bit in (("page", sa.SA_DEV_INDEX), ("range", sa.SA_DEV_INDEX), ("negative", sa.SA_DEV_INDEX), ("order", sa.SA_DEV_ORDER),
                          ("gap", sa.SA_DEV_ORDER)):
            if not q8 and what in ("order", "gap"):
                continue
            x = append_inputs([70, 30], [4, 4], T, Hq, d, D_I, 128, False, q8, 64, False, True, seed=9)
            if what == "page":
                x["pt"][0, 1] = x["pool"]
            elif what == "range":
                x["nv"][1] = x["pt"].shape[1] * 64 + 1
            elif what == "negative":
                x["nv"][1] = -5
            elif what == "order":
                x["nv"][2] = x["nv"][1]
            else:
                x["nv"][1] = 0
            y = run_append(sa, x, T, Hq, d, D_I, 128, False, q8, 64, False)
            assert int(y["status"].item()) == bit, what
            if q8 or what == "page":   # nothing of sequence 0 is written
                mine = x["pt"][0, :2].long()
                keep = (mine[mine < x["pool"]][:, None] * 64 + torch.arange(64)).view(-1)
                for n in ("kc", "vc", "kIc"):
                    assert torch.equal(y[n].cpu()[keep], x[n][keep]), (what, n)
            # the other sequence is appended as ever
            s = ref.slot_of(x["pt"], 0, 1, 29)
            assert torch.equal(y["kIc"].cpu()[s], x["kI"][7])


# ---------------------------------------------------------------- attention
def filled_cache(n, d, sb, g, spread=2):
    codes = torch.randn(n, d, generator=g).mul(60).clamp(-448, 448).to(ref.E4M3).view(torch.uint8)
    scale = torch.exp2(torch.randint(-6 - spread, -6 + spread, (n // sb,), generator=g).float()) * (1 + torch.rand(n // sb, generator=g))
    return codes, scale


def attention_inputs(lens, news, T, Hq, d, K, W, sb, paged, seed):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    x = dict(nv=ref.rows_of(lens, news, T), S_max=max(64, -(-max(lens) // 64) * 64))
    x["pt"], x["pool"] = ref.paged_table(lens, g) if paged else (None, 0)
    n = x["pool"] * 64 if paged else B * x["S_max"]
    x["kc"], x["ks"] = filled_cache(n, d, sb, g)
    x["vc"], x["vs"] = filled_cache(n, d, sb, g)
    x["q"] = torch.randn(B * T, Hq, d, generator=g).bfloat16()
    topk = torch.full((B * T, K), -1, dtype=torch.int32)
    for r in range(B * T):
        n_r = int(x["nv"][r])
        pick = torch.randperm(n_r, generator=g)[:K].sort().values
        topk[r, :len(pick)] = pick.to(torch.int32)
    x["topk"] = topk
    return x


def run_attention(sa, x, T, Hq, d, K, W, sb, lse=True, y=None):
    R, B = x["nv"].numel(), x["nv"].numel() // T
    y = y or {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    out, status = torch.full((R, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda"), status_word()
    ls = torch.full((R, Hq), 3.0, device="cuda") if lse else None
    pt = y.get("pt")
    sa.sa_sparse_attn_q8(y["q"], y["kc"], y["vc"], y["ks"], y["vs"], sb, pt, pt.shape[1] if pt is not None else 0, x["pool"], 64,
                         x["S_max"], y["nv"], y["topk"] if K else None, K, W, B, T, Hq, d, d ** -0.5, out, ls, status)
    torch.cuda.synchronize()
    return out.cpu(), ls.cpu() if lse else None, int(status.item())


def check_attention(x, got, T, K, W, sb, scale=None):
    out, lse, _ = got
    d = x["q"].shape[-1]
    want, wl, tol, tl, sizes = ref.attention(x["q"], x["kc"], x["vc"], x["ks"], x["vs"], sb, x["pt"], x["S_max"], x["nv"],
                                             x["topk"] if K else None, W, T, scale or d ** -0.5)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), "out off by %.3g where %.3g is allowed" % (float(err.max()), float(tol.flatten()[(err - tol).argmax()]))
    for r, n in enumerate(sizes):
        if n == 0:
            assert (out[r] == 0).all() and (lse is None or (lse[r] == -math.inf).all())
        elif lse is not None:
            e = (lse[r].double() - wl[r]).abs()
            assert (e <= tl[r]).all(), "lse off by %.3g where %.3g is allowed" % (float(e.max()), float(tl[r].min()))
    return sizes


ATTENTIONS = [
    # lens, news, T, Hq, d, K, W, sb, paged
    ([1], [1], 1, 1, 128, 8, 4, 64, True),
    ([1, 2, 300], [1, 1, 1], 1, 16, 128, 64, 32, 64, True),
    ([700, 64, 2000], [1, 1, 1], 1, 64, 128, 256, 64, 32, True),
    ([5000], [1], 1, 64, 128, 2048, 512, 64, False),
    ([3000, 129], [1, 1], 1, 33, 64, 1000, 1, 16, False),
    ([257, 385, 511], [4, 4, 4], 4, 32, 128, 128, 128, 8, True),
    ([100, 30, 64], [37, 0, 20], 37, 5, 64, 64, 32, 16, True),
    ([40], [40], 40, 48, 128, 16, 0, 1, True),
    ([300], [9], 9, 17, 128, 77, 45, 64, False),
    ([9000], [3], 3, 64, 64, 4096, 512, 64, True),
    ([1500, 1800], [90, 90], 90, 16, 128, 200, 56, 64, True),
    ([260], [260], 260, 3, 128, 0, 129, 32, False),
]


@pytest.mark.parametrize("case", range(len(ATTENTIONS)))
def test_attention(sa, case):
    lens, news, T, Hq, d, K, W, sb, paged = ATTENTIONS[case]
    x = attention_inputs(lens, news, T, Hq, d, K, W, sb, paged, seed=case)
    got = run_attention(sa, x, T, Hq, d, K, W, sb, lse=case % 4 != 1)
    assert got[2] == 0
    check_attention(x, got, T, K, W, sb)


@pytest.mark.parametrize("Hq,T", [(16, 1), (64, 1), (16, 200), (64, 40)])
def test_attention_growing_scores_and_uneven_scales(sa, Hq, T):
    """Scores that grow along the keys (the running maximum is raised tile by tile), value scales 2^60 apart, and scales
    beyond the range that count as its ends."""
    d, K, W, sb, L = 128, 512, 64, 16, 1200
    x = attention_inputs([L], [T], T, Hq, d, K, W, sb, True, seed=Hq + T)
    g = torch.Generator().manual_seed(3)
    order = [ref.slot_of(x["pt"], 0, 0, p) // sb for p in range(0, L, sb)]
    for i, blk in enumerate(order):
        x["ks"][blk] = 2.0 ** (-10 + 5 * i / len(order))
        x["vs"][blk] = 2.0 ** float(torch.randint(-30, 31, (1,), generator=g))
    x["vs"][order[3]], x["vs"][order[5]], x["ks"][order[7]] = 0.0, 1e-30, 0.0
    got = run_attention(sa, x, T, Hq, d, K, W, sb)
    assert got[2] == 0
    check_attention(x, got, T, K, W, sb)


@pytest.mark.parametrize("Hq,T,order", [(16, 1, 1), (64, 160, 1), (64, 1, -1), (16, 160, -1), (33, 2, 0)])
def test_attention_of_huge_scores(sa, Hq, T, order):
    """Scores up to 10^9, 10^30 and 10^36 of which each is 1.2 times the next: the largest takes the whole weight, however
    coarse fp32 is there.  Every key has the same codes, so a head's largest score is the largest or the smallest scale's."""
    d, K, sb, L = 128, 400, 1, 400
    for up in (-20, 50, 70):
        x = attention_inputs([L], [T], T, Hq, d, K, 0, sb, True, seed=Hq + T)
        g = torch.Generator().manual_seed(12)
        x["kc"][:] = x["kc"][0].clone()
        x["q"] = (x["q"].double() * 2.0 ** up).bfloat16()
        step = torch.arange(L) if order > 0 else torch.arange(L).flip(0) if order < 0 else torch.randperm(L, generator=g)
        slots = torch.tensor([ref.slot_of(x["pt"], 0, 0, p) for p in range(L)])
        x["ks"][slots] = (2.0 ** -60 * 1.2 ** step.double()).float()
        out, lse, st = run_attention(sa, x, T, Hq, d, K, 0, sb)
        assert st == 0 and torch.isfinite(out).all()
        ks, code, checked = x["ks"][slots].double(), ref.of_e4m3(x["kc"][0]), 0
        s = (x["q"].double() @ code) * d ** -0.5   # [rows, heads]
        for r in range(T):
            two, at = (s[r][:, None] * ks[None, :int(x["nv"][r])]).topk(2)
            clear = two[:, 0] - two[:, 1] > 60   # (the others are near ties: not this test's concern)
            want = ref.of_e4m3(x["vc"][slots[at[:, 0]]]) * x["vs"][slots[at[:, 0]]].double()[:, None]
            # P's two parts and the output's rounding, 2^-8 each, their product, fp32 sums, and e^-60 of the others
            err = (out[r].double() - want).abs()
            assert (err <= (2.0 ** -7 + 2.0 ** -12) * want.abs() + 1e-9)[clear].all(), (up, r)
            # q's small values are off by 2^-18 of the largest, the fp32 score by 2^-20
            dx = x["q"][r].double().abs().max() * 2.0 ** -18 * code.abs().sum() * d ** -0.5 * ks[at[:, 0]]
            assert ((lse[r].double() - two[:, 0]).abs() <= dx + 2.0 ** -20 * two[:, 0].abs() + 1e-3)[clear].all(), (up, r)
            checked += int(clear.sum())
        assert checked > (0 if up < 70 else 0.9 * T * Hq)


@pytest.mark.parametrize("T", [1, 150])
def test_attention_rows_without_keys(sa, T):
    """W = 0 and rows whose top-K is empty, beside padding rows and full ones."""
    Hq, d, K, sb = 8, 128, 40, 64
    x = attention_inputs([300, 290, 200], [T, T, T], T, Hq, d, K, 0, sb, True, seed=2)
    x["topk"][0] = -1
    x["topk"][2 * T - 1] = -1
    x["nv"][2 * T] = 0
    got = run_attention(sa, x, T, Hq, d, K, 0, sb)
    assert got[2] == 0
    sizes = check_attention(x, got, T, K, 0, sb)
    assert sizes[0] == sizes[2 * T - 1] == sizes[2 * T] == 0


@pytest.mark.parametrize("T", [1, 160])
def test_attention_never_reads_what_is_not_selected(sa, T):
    """NaN codes in every slot that no row selects, and in the rows behind the last token: no trace of them."""
    Hq, d, K, W, sb, L = 20, 128, 70, 33, 64, 400
    x = attention_inputs([L], [T], T, Hq, d, K, W, sb, True, seed=4)
    used = torch.zeros(len(x["kc"]), dtype=torch.bool)
    for r in range(T):
        p = int(x["nv"][r]) - 1
        keys = [e for e in x["topk"][r].tolist() if 0 <= e <= p - W] + list(range(max(0, p - W + 1), p + 1))
        used[torch.tensor([ref.slot_of(x["pt"], 0, 0, s) for s in keys])] = True
    x["kc"][~used], x["vc"][~used] = 0x7F, 0xFF
    got = run_attention(sa, x, T, Hq, d, K, W, sb)
    assert got[2] == 0
    check_attention(x, got, T, K, W, sb)


def test_attention_keeps_nan_to_the_rows_that_select_it(sa):
    Hq, d, K, W, sb, T = 16, 128, 64, 8, 64, 150
    x = attention_inputs([500], [T], T, Hq, d, K, W, sb, True, seed=5)
    bad = 40   # a position that some rows select
    x["vc"][ref.slot_of(x["pt"], 0, 0, bad)] = 0x7F
    out, _, st = run_attention(sa, x, T, Hq, d, K, W, sb)
    has = (x["topk"] == bad).any(1)
    assert st == 0 and has.any() and not has.all()
    assert torch.isnan(out[has]).all() and torch.isfinite(out[~has]).all()


@pytest.mark.parametrize("Hq,T", [(5, 1), (64, 1), (33, 200)])
def test_attention_keeps_odd_queries_to_their_heads(sa, Hq, T):
    """Infinite and NaN queries make their own head's output NaN and no other; a row of zeros weighs its keys alike, and
    the smallest numbers count."""
    d, K, W, sb = 128, 96, 20, 64
    x = attention_inputs([400], [T], T, Hq, d, K, W, sb, True, seed=20 + Hq)
    x["q"][0, 1, 7], x["q"][0, 3, 100] = math.inf, math.nan
    if T > 1:
        x["q"][1] = 0
        x["q"][2] = 2.0 ** -133   # bf16's smallest
        x["q"][3, :, ::2] *= 2.0 ** -100
        x["q"][4, 0] = -math.inf
    got = run_attention(sa, x, T, Hq, d, K, W, sb)
    assert got[2] == 0
    odd = ~torch.isfinite(x["q"]).all(-1)
    assert torch.isnan(got[0][odd]).all() and torch.isnan(got[1][odd]).all() and odd.sum() == 2 + (T > 1)
    z = dict(x, q=torch.where(odd[..., None], torch.zeros_like(x["q"]), x["q"]))
    plain = run_attention(sa, z, T, Hq, d, K, W, sb)
    out, lse = got[0].clone(), got[1].clone()
    out[odd], lse[odd] = plain[0][odd], plain[1][odd]
    check_attention(z, (out, lse, 0), T, K, W, sb)


def test_attention_of_many_rows_of_which_few_are_there(sa):
    """200,000 rows, all but some of them padding."""
    B, T, Hq, d, K, W, sb = 50, 4000, 3, 64, 12, 5, 16
    g = torch.Generator().manual_seed(31)
    lens = torch.randint(20, 90, (B,), generator=g).tolist()
    x = attention_inputs(lens, [1 + b % 3 if b % 7 == 0 else 0 for b in range(B)], T, Hq, d, 0, W, sb, True, seed=31)
    topk = torch.full((B * T, K), -1, dtype=torch.int32)
    for r in torch.nonzero(x["nv"]).flatten().tolist():
        topk[r, :6] = torch.randperm(int(x["nv"][r]), generator=g)[:6].sort().values.to(torch.int32)
    x["topk"] = topk
    out, lse, st = run_attention(sa, x, T, Hq, d, K, W, sb)
    there = x["nv"] > 0
    assert st == 0 and (out[~there] == 0).all() and (lse[~there] == -math.inf).all()
    for b in range(0, B, 7):
        rows = slice(b * T, b * T + 4)
        want, wl, tol, tl, _ = ref.attention(x["q"][rows], x["kc"], x["vc"], x["ks"], x["vs"], sb, x["pt"][b:b + 1], x["S_max"],
                                             x["nv"][rows], topk[rows], W, 4, d ** -0.5)
        assert ((out[rows].double() - want).abs() <= tol).all()


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import fine_grained_top_b200 as sa
from tests import test_cache_ops_gpu as t
for T, Hq in ((1, 64), (1, 16), (300, 32)):
    x = t.attention_inputs([900] * 2, [T] * 2, T, Hq, 64, 256, 64, 64, True, seed=40)
    y = {{n: v.cuda() for n, v in x.items() if isinstance(v, torch.Tensor)}}
    out, lse = torch.zeros(2 * T, Hq, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2 * T, Hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sa_sparse_attn_q8(y["q"], y["kc"], y["vc"], y["ks"], y["vs"], 64, y["pt"], y["pt"].shape[1], x["pool"], 64, 0, y["nv"],
                             y["topk"], 256, 64, 2, T, Hq, 64, 0.125, out, lse)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    eager = t.run_attention(sa, x, T, Hq, 64, 256, 64, 64)
    assert torch.equal(out.cpu(), eager[0]) and torch.equal(lse.cpu(), eager[1])
print("same")
"""


def test_a_process_whose_first_calls_are_captured(sa):
    import subprocess
    import sys

    from tests.conftest import ROOT
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=str(ROOT))], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("T", [1, 170])
def test_attention_reports_bad_entries(sa, T):
    """A page id outside of the pool, a top-K entry behind the row's position, an unsorted row and a length beyond the
    cache: reported, skipped, and the other rows are right."""
    Hq, d, K, W, sb = 16, 128, 64, 16, 64
    x = attention_inputs([640, 640], [T, T], T, Hq, d, K, W, sb, True, seed=6)
    good = run_attention(sa, x, T, Hq, d, K, W, sb)
    assert good[2] == 0

    def variant(change):
        z = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
        change(z)
        return z, run_attention(sa, z, T, Hq, d, K, W, sb)

    last = 2 * T - 1
    z, got = variant(lambda z: z["pt"][1].__setitem__(2, z["pool"] + 3))
    assert got[2] == sa.SA_DEV_INDEX and torch.equal(got[0][:T], good[0][:T])
    # the bad page's keys are left out: the same as a top-K without them
    w = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    for r in range(T, 2 * T):
        e = [v for v in w["topk"][r].tolist() if v >= 0 and not 128 <= v < 192]
        w["topk"][r] = torch.tensor(e + [-1] * (K - len(e)), dtype=torch.int32)
    check_attention(w, got, T, K, W, sb)
    z, got = variant(lambda z: z["topk"][last].__setitem__(K - 1, 5000))
    assert got[2] == sa.SA_DEV_INDEX and torch.equal(got[0][:last], good[0][:last])
    z, got = variant(lambda z: z["topk"][last].__setitem__(slice(0, 2), z["topk"][last, :2].flip(0)))
    assert got[2] == sa.SA_DEV_ORDER and torch.equal(got[0][:last], good[0][:last])
    for n in (641, -1, 2 ** 30):
        z, got = variant(lambda z: z["nv"].__setitem__(last, n))
        assert got[2] == sa.SA_DEV_INDEX and torch.equal(got[0][:last], good[0][:last])
        assert (got[0][last] == 0).all() and (got[1][last] == -math.inf).all()


def test_attention_rows_beyond_32_bit_offsets(sa):
    """A pool of 34.6 million tokens: the byte offsets of its last pages pass 2^32."""
    d, K, W, sb, T, Hq, L = 128, 100, 30, 64, 2, 16, 700
    x = attention_inputs([L], [T], T, Hq, d, K, W, sb, True, seed=7)
    n_pages = 540_000
    y = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    for s in "kv":
        big = torch.empty(n_pages * 64, d, dtype=torch.uint8, device="cuda")
        big[-x["pool"] * 64:] = y[s + "c"]
        scales = torch.ones(n_pages * 64 // sb, device="cuda")
        scales[-x["pool"] * 64 // sb:] = y[s + "s"]
        y[s + "c"], y[s + "s"] = big, scales
    y["pt"] = y["pt"] + (n_pages - x["pool"])
    small = run_attention(sa, x, T, Hq, d, K, W, sb)
    large = run_attention(sa, dict(x, pool=n_pages), T, Hq, d, K, W, sb, y=y)
    assert small[2] == large[2] == 0 and torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    # and the append writes there
    st, k = status_word(), torch.randn(1, d, device="cuda").bfloat16()
    nv = torch.tensor([L], dtype=torch.int32, device="cuda")
    args = (None, 0, None, k, d, k, d, None, 0, nv, y["pt"], y["pt"].shape[1], n_pages, 64, 0, 1, 1, 0, d, 0, None, 0, 0)
    before = [int(y[s + "c"][:1000].long().sum()) for s in "kv"]
    sa.sa_cache_append_q8(*args, y["kc"], y["vc"], y["ks"], y["vs"], sb, None, 0, st)
    slot = int(y["pt"][0, (L - 1) // 64]) * 64 + (L - 1) % 64
    val = y["kc"][slot].view(ref.E4M3).float() * y["ks"][slot // sb]
    # e4m3's half step, and among its subnormals 2^-10 of the scale
    assert ((val - k[0].float()).abs() <= 2.0 ** -4 * k[0].float().abs() + 2.0 ** -10 * y["ks"][slot // sb]).all()
    assert int(st.item()) == 0 and before == [int(y[s + "c"][:1000].long().sum()) for s in "kv"]


def test_attention_is_the_same_every_time(sa):
    x = attention_inputs([3000, 2500], [40, 40], 40, 64, 128, 600, 100, 64, True, seed=8)
    first = run_attention(sa, x, 40, 64, 128, 600, 100, 64)
    for _ in range(3):
        again = run_attention(sa, x, 40, 64, 128, 600, 100, 64)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------- run together
def together(q8, T, seed, paged=True, index_fp8=False):
    from fine_grained_top_b200.pipeline import DecodePlan, KVCache
    B, Hq, d, H_I, D_I, K, W, sb = 3, 16, 128, 4, 64, 64, 16, 32
    g = torch.Generator().manual_seed(seed)
    lens = [200, 77, 330]
    pt, pool = ref.paged_table([n + 64 for n in lens], g)
    cache = KVCache(B, d, D_I, S_max=512, paged=paged, max_pages=pt.shape[1], pool_pages=pool, q8=q8, scale_block=sb,
                    index_fp8=index_fp8)
    plan = DecodePlan(B, Hq, d, H_I, D_I, K, W, T=T, cache=cache)
    return B, Hq, d, H_I, D_I, K, W, sb, g, lens, pt.cuda() if paged else None, cache, plan


@pytest.mark.parametrize("q8,T,paged,index_fp8", [(True, 1, True, False), (True, 3, True, True), (False, 1, True, False),
                                                  (True, 2, False, False), (False, 1, False, True)])
def test_prompt_then_steps(sa, q8, T, paged, index_fp8):
    """A prompt enters the cache, then steps of T tokens: each step's attention equals the 64-bit attention over the values
    the cache then holds, with the rotated queries and the selection that the indexer made."""
    B, Hq, d, H_I, D_I, K, W, sb, g, lens, pt, cache, plan = together(q8, T, 1, paged, index_fp8)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).bfloat16().cuda()  # noqa: E731
    top = max(lens)
    cache.append(None, bf(B * top, d), bf(B * top, d), ints(B * top, D_I), ref.rows_of(lens, lens, top).cuda(), top, pt)
    held = list(lens)
    for step in range(4):
        held = [n + T for n in held]
        nv = ref.rows_of(held, [T] * B, T)
        qI = ints(B * T, H_I, D_I)
        if index_fp8:
            q8b = torch.empty(qI.shape, dtype=torch.uint8, device="cuda")
            sa.sa_convert_e4m3(qI, q8b, qI.numel())
            qI = q8b
        x = dict(q=bf(B * T, Hq, d), k=bf(B * T, d), v=bf(B * T, d), kI=ints(B * T, D_I), qI=qI,
                 w=torch.randint(0, 4, (B * T, H_I), generator=g).bfloat16().cuda(), lengths=nv.cuda(), page_table=pt)
        for _, fn in plan.stages(x):
            fn()
        torch.cuda.synchronize()
        assert int(plan.dev_status.item()) == 0
        topk = plan.topk.cpu()
        for r in range(B * T):   # a full top-K among the row's own tokens
            e = topk[r][topk[r] >= 0]
            assert len(e) == min(K, int(nv[r])) and int(e.max()) < int(nv[r])
        q = plan.q_rot.cpu()
        flat = lambda t: t.cpu().view(-1, t.shape[-1])  # noqa: E731
        if q8:
            want, wl, tol, tl, _ = ref.attention(q, flat(cache.k), flat(cache.v), cache.k_scale.cpu().view(-1),
                                                 cache.v_scale.cpu().view(-1), sb, None if pt is None else pt.cpu(), cache.S_max,
                                                 nv, topk, W, T, plan.scale)
            assert ((plan.out.cpu().double() - want).abs() <= tol).all() and ((plan.lse.cpu().double() - wl).abs() <= tl).all()
        else:
            kf, vf = flat(cache.k).double(), flat(cache.v).double()
            for b in range(B):
                p = int(nv[b]) - 1
                keys = [e for e in topk[b].tolist() if 0 <= e <= p - W] + list(range(max(0, p - W + 1), p + 1))
                s = torch.tensor([ref.slot_of(None if pt is None else pt.cpu(), cache.S_max, b, i) for i in keys])
                w = torch.softmax(q[b].double() @ kf[s].T * plan.scale, -1)
                # probabilities and outputs are rounded to bf16, 2^-8 each; twice that for the fp32 softmax's slack
                tol = 2.0 ** -7 * (w @ vf[s].abs())
                assert ((plan.out[b].cpu().double() - w @ vf[s]).abs() <= tol).all()


def test_captured_step_replays(sa):
    """A whole step in a CUDA graph, replayed with new tokens and lengths, equals the same steps run eagerly; two graphs of
    two plans share nothing, and a step on another stream gives the same."""
    results = []
    for mode in ("eager", "graph", "stream"):
        B, Hq, d, H_I, D_I, K, W, sb, g, lens, pt, cache, plan = together(True, 1, 2)
        bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
        top = max(lens)
        cache.append(None, bf(B * top, d), bf(B * top, d), bf(B * top, D_I), ref.rows_of(lens, lens, top).cuda(), top, pt)
        x = dict(q=bf(B, Hq, d), k=bf(B, d), v=bf(B, d), kI=bf(B, D_I), qI=bf(B, H_I, D_I), w=bf(B, H_I),
                 lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), page_table=pt)
        stream = torch.cuda.Stream() if mode == "stream" else None
        stages = plan.stages(x, stream)
        graph = None
        outs = []
        for step in range(5):
            fresh = dict(q=bf(B, Hq, d), k=bf(B, d), v=bf(B, d), kI=bf(B, D_I), qI=bf(B, H_I, D_I), w=bf(B, H_I))
            for n, t in fresh.items():
                x[n].copy_(t)
            x["lengths"] += 1
            if mode == "graph" and step == 1:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    for _, fn in stages:
                        fn()
            if graph is not None:
                graph.replay()
            elif stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
                for _, fn in stages:
                    fn()
                torch.cuda.current_stream().wait_stream(stream)
            else:
                for _, fn in stages:
                    fn()
            torch.cuda.synchronize()
            outs.append((plan.out.clone(), plan.lse.clone(), cache.k.clone(), cache.k_scale.clone()))
        assert int(plan.dev_status.item()) == 0
        results.append(outs)
    for outs in results[1:]:
        for a, b in zip(results[0], outs):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_two_calls_at_once(sa):
    """The same attention on two streams at once, few rows (clusters) and many rows (a CTA each)."""
    xs = [attention_inputs([3000] * 2, [1, 1], 1, 64, 128, 512, 64, 64, True, seed=10),
          attention_inputs([900] * 2, [180, 180], 180, 16, 128, 128, 32, 64, True, seed=11)]
    shapes = [(1, 64, 128, 512, 64, 64), (180, 16, 128, 128, 32, 64)]
    alone = [run_attention(sa, x, *s) for x, s in zip(xs, shapes)]
    ys = [{n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)} for x in xs]
    streams, outs = [torch.cuda.Stream() for _ in range(4)], []
    torch.cuda.synchronize()
    for i, st in enumerate(streams):
        x, y, (T, Hq, d, K, W, sb) = xs[i % 2], ys[i % 2], shapes[i % 2]
        out, lse = torch.zeros(x["nv"].numel(), Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(x["nv"].numel(), Hq, device="cuda")
        torch.cuda.synchronize()
        outs.append((out, lse))
        for _ in range(3):
            sa.sa_sparse_attn_q8(y["q"], y["kc"], y["vc"], y["ks"], y["vs"], sb, y["pt"], y["pt"].shape[1], x["pool"], 64, 0, y["nv"],
                                 y["topk"], K, W, 2, T, Hq, d, d ** -0.5, out, lse, None, st)
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(out.cpu(), alone[i % 2][0]) and torch.equal(lse.cpu(), alone[i % 2][1])
