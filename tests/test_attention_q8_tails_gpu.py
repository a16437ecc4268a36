"""GPU tests of the attention over the 8-bit cache where one key takes most of a
head's weight and hardly any of its value (an attention sink): the output is
then made by the many keys far below it, and every one of them has to count.

Tolerances: the output's rounding to bf16 is off by 2^-8 of it.  A probability
in fp16 is off by 2^-11 of its value; held so that a head's largest is at least
2^7.75, one 14 nats (20.2 bits) below is 2^-12.5 and its own rounding within
2^-12.5 of it, so that 2^-10 of sum w|v| covers both however many keys there
are.  The scores' slack is that of tests/cache_reference.py."""

import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    import fine_grained_top_b200 as m
    return m


def sink_inputs(T, Hq, d, n, sb, dev, share, at, seed):
    """One sequence of n cached tokens, T rows that see all but the last T - 1 - t of them; key `at` lies 6 to 14 nats
    above the others' mean, by head, whose scores have the standard deviation `dev` (0: equal); its value is `share` of
    theirs.  Key and value scales are the same for the sink and its neighbours' block."""
    g = torch.Generator().manual_seed(seed)
    kc = torch.randn(n, d, generator=g).mul(60)
    vc = torch.randn(n, d, generator=g).mul(100) + 40 * torch.randn(d, generator=g)
    kc[:, 0] = 0
    kc[at] = 0
    kc[at, 0] = 448
    vc[at] *= share
    ks, vs = 2.0 ** -8, 2.0 ** -7
    q = torch.randn(T, Hq, d, generator=g) * dev / (60 * ks * (d - 1) ** 0.5 * d ** -0.5)
    q[..., 0] = torch.linspace(6, 14, Hq) / (448 * ks * d ** -0.5)
    x = dict(q=q.bfloat16(), kc=kc.clamp(-448, 448).to(ref.E4M3).view(torch.uint8),
             vc=vc.clamp(-448, 448).to(ref.E4M3).view(torch.uint8), ks=torch.full((n // sb,), ks), vs=torch.full((n // sb,), vs))
    x["nv"] = torch.arange(n - T + 1, n + 1, dtype=torch.int32)
    return x


def run(sa, x, B, T, K, W, sb, topk=None, scale=None):
    R, Hq, d = x["q"].shape
    y = {n: t.cuda() for n, t in x.items()}
    n = len(x["kc"]) // B
    out, lse = torch.full((R, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((R, Hq), 3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sa.sa_sparse_attn_q8(y["q"], y["kc"], y["vc"], y["ks"], y["vs"], sb, None, 0, 0, 64, n, y["nv"],
                         topk.cuda() if K else None, K, W, B, T, Hq, d, scale or d ** -0.5, out, lse, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.cpu().double(), lse.cpu().double()


def want(x, sb, keys, r, scale):
    """The row's exact output and lse, sum w|v| and the relative slack of its weights."""
    kc, vc, q = ref.of_e4m3(x["kc"][keys]), ref.of_e4m3(x["vc"][keys]), x["q"][r].double()
    ks, vs = x["ks"][keys // sb].double(), x["vs"][keys // sb].double()
    s = (q @ kc.T) * ks * scale
    z = torch.logsumexp(s, -1)
    w = torch.exp(s - z[:, None]) * vs
    dx = (q.abs().max() * 2.0 ** -10 / 224 * kc.abs().sum(-1) * ks * abs(scale)).max()
    mag = ((q.abs() @ kc.abs().T) * ks * abs(scale)).max()
    rel = float(dx + mag * 2.0 ** -22) * 2 + 2.0 ** -18 + len(keys) * 2.0 ** -24
    return w @ vc, z, w @ vc.abs(), rel


@pytest.mark.parametrize("Hq,d,T,at", [(16, 128, 1, 3), (5, 64, 1, 700), (64, 128, 1, 2559), (32, 128, 3, 1300),
                                       (16, 128, 300, 100), (64, 128, 300, 1500), (33, 64, 320, 5), (20, 128, 310, 2200)])
@pytest.mark.parametrize("dev,share", [(0.0, 0.0), (0.3, 0.0), (1.0, 0.02), (2.0, 0.05)])
def test_the_keys_below_a_sink_count(sa, Hq, d, T, at, dev, share):
    n, sb = 2560, 64
    W = n   # every key, by the window: the rows see n - T + 1 .. n of them
    x = sink_inputs(T, Hq, d, n, sb, dev, share, min(at, n - T), seed=Hq + T)
    out, lse = run(sa, x, 1, T, 0, W, sb)
    for r in sorted({0, T // 2, T - 1}):
        o, z, aw, rel = want(x, sb, torch.arange(int(x["nv"][r])), r, d ** -0.5)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -10 + rel) * aw
        err = (out[r] - o).abs()
        assert (err <= tol).all(), "off by %.3g of sum w|v|" % float((err / aw).max())
        assert ((lse[r] - z).abs() <= rel + 2.0 ** -22 * z.abs()).all()


@pytest.mark.parametrize("Hq,d", [(16, 128), (64, 64)])
def test_a_row_is_the_same_in_small_and_large_steps(sa, Hq, d):
    """A row split over a cluster and the same row as one of 400: both within the tolerance of the exact one, hence within
    twice that of each other."""
    n, sb, K = 2560, 64, 2000
    x = sink_inputs(1, Hq, d, n, sb, 0.3, 0.0, 900, seed=3)
    g = torch.Generator().manual_seed(4)
    pick = torch.randperm(n, generator=g)[:K].sort().values
    if 900 not in pick:
        pick[int((pick < 900).sum())] = 900
    topk = pick.to(torch.int32)[None]
    big = dict(x, q=x["q"].expand(400, -1, -1).contiguous(), nv=x["nv"].expand(400).contiguous())
    one = run(sa, x, 1, 1, K, 0, sb, topk)
    many = run(sa, big, 1, 400, K, 0, sb, topk.expand(400, -1).contiguous())
    o, z, aw, rel = want(x, sb, pick, 0, d ** -0.5)
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -10 + rel) * aw
    assert ((one[0][0] - o).abs() <= tol).all() and ((many[0] - o).abs() <= tol).all()
    assert ((one[1][0] - z).abs() <= rel + 2.0 ** -22 * z.abs()).all()
    assert (many[0] == many[0][0]).all() and (many[1] == many[1][0]).all()


def test_equal_keys_far_below_a_sink_share_its_tail(sa):
    """Every key but the sink has the same code rows: the output is their value times their weight, to the rounding."""
    n, sb, d, Hq = 8192, 64, 128, 8
    x = sink_inputs(1, Hq, d, n, sb, 0.0, 0.0, 77, seed=9)
    x["vc"][:] = x["vc"][0].clone()
    x["vc"][77] = 0
    out, _ = run(sa, x, 1, 1, 0, n, sb)
    o, _, aw, rel = want(x, sb, torch.arange(n), 0, d ** -0.5)
    assert ((out[0] - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -10 + rel) * aw).all()


@pytest.mark.parametrize("Hq,T", [(16, 1), (64, 1), (16, 300), (40, 300)])
@pytest.mark.parametrize("order", ["small first", "large first", "in turn"])
def test_keys_of_the_smallest_value_scale_weigh_as_much_as_any(sa, Hq, T, order):
    """Value scales at both ends of their range (2^64 and 2^-64) under scores of one size: the small ones' keys count in
    the row sum, whichever the row meets first, in one tile, in tiles apart and in the parts of a cluster."""
    n, sb, d, W = 1280, 64, 128, 1280
    x = sink_inputs(T, Hq, d, n, sb, 1.0, 1.0, 0, seed=50 + T)
    x["q"][..., 0] = 0   # no sink
    blocks = n // sb
    small = {"small first": torch.arange(blocks) < blocks // 2, "large first": torch.arange(blocks) >= blocks // 2,
             "in turn": torch.arange(blocks) % 2 == 1}[order]
    x["vs"] = torch.where(small, 2.0 ** -64, 2.0 ** 64).float()
    out, lse = run(sa, x, 1, T, 0, W, sb)
    for r in sorted({0, T // 2, T - 1}):
        o, z, aw, rel = want(x, sb, torch.arange(int(x["nv"][r])), r, d ** -0.5)
        assert ((lse[r] - z).abs() <= rel + 2.0 ** -22 * z.abs()).all(), float((lse[r] - z).abs().max())
        assert ((out[r] - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -10 + rel) * aw).all()


@pytest.mark.parametrize("Hq,d,T,paged_tiles", [(16, 128, 1, 1), (64, 128, 1, 9), (32, 128, 3, 4), (16, 64, 300, 3), (64, 128, 300, 5),
                                                (33, 128, 320, 2)])
def test_a_head_of_large_queries_leaves_the_others_their_precision(sa, Hq, d, T, paged_tiles):
    """One head's queries are 2^20 times the others' (and one head is all zeros): the others' outputs and lse are as exact
    as without it.  Rows in which heads lie 2^5 apart, or in which every head is large, go with them."""
    n, sb = 128 * paged_tiles, 64
    n = max(n, (T + 63) // 64 * 64)
    x = sink_inputs(T, Hq, d, n, sb, 1.0, 1.0, 0, seed=70 + T)
    q = x["q"].double()
    q[..., 0] = 0
    q[:, 1] *= 2.0 ** 20
    q[:, 2] = 0
    q[T // 2, 1] *= 2.0 ** -15
    q[T - 1, 3:] *= 2.0 ** 20 if T > 1 else 1.0
    x["q"] = q.bfloat16()
    out, lse = run(sa, x, 1, T, 0, n, sb)
    for r in sorted({0, T // 2, T - 1}):
        keys = torch.arange(int(x["nv"][r]))
        for h in [0, 2, 4, Hq - 1]:
            if q[r, h].abs().max() > 100:
                continue   # a head of large scores
            alone = dict(x, q=x["q"][:, h:h + 1])   # its own slack, not the row's
            o, z, aw, rel = want(alone, sb, keys, r, d ** -0.5)
            assert ((lse[r, h:h + 1] - z).abs() <= rel + 2.0 ** -22 * z.abs()).all(), (r, h)
            assert ((out[r, h:h + 1] - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -10 + rel) * aw).all(), (r, h)
