"""GPU: the norm with the residual's addition (forward, 8-bit output, backward)
and rows to 8 bits and back, against their plain forms in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24; half = half a step of the
output type, 2^-8 bf16, 2^-24 fp32):
  h      the same bits (one fp32 sum, one rounding).
  rstd   a sum of d squares (all positive) in fp32 by partial sums of at most
         d / 64 + 64 terms, halved by the root: (d / 64 + 64) u relative.
  y      rstd's error, two products and the output's rounding, relative to y.
  q, s   from a given matrix: the same integers and the same scales.  From the
         norm: s within y's error of the plain one, and q s within s / 2 of
         the plain y plus y's error.
  dx     the two terms' products (8 u of each), the dot product's error
         (d / 64 + 64) u sum_j |w dy h| scaled by |h| rstd^3 / d, one rounding.
  dw     (T + 8) u sum_t |dy h rstd| (any order of at most T terms).
"""
import pytest
import torch

import rows8_ref as R
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half(dt):
    return torch.finfo(dt).eps / 2


def draw(seed, T, d, dt, spread=True):
    g = torch.Generator().manual_seed(seed)
    x, res, dy, dres = (torch.randn(T, d, generator=g) for _ in range(4))
    if spread and d > 3:
        res[:, d // 3] *= 40.0
    w = 1 + 0.2 * torch.randn(d, generator=g)
    return [t.to(dt) for t in (x, res, w, dy, dres)]


def up(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def within(got, ref, bound, what):
    got = got.cpu().double()
    assert got.shape == ref.shape, what
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert (off <= bound).all(), (f"{what}: {int((off > bound).sum())} of {off.numel()} off, worst "
                                  f"{float((off / bound.clamp_min(1e-300)).max()):.2f}x the bound")


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 8), (5, 33), (4, 63), (7, 130), (16, 512), (33, 1027),
          (9, 2048), (6, 5119), (3, 8192), (2, 16384), (2, 16387), (2, 28672), (1, 32768),
          (2, 32775), (1, 70001)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rmsnorm_matches_plain_form(T, d, dt):
    for group, with_res in ((0, True), (128, False), (32, True), (512, True)):
        say("rmsnorm", T, d, dt, group, with_res)
        x, res, w, _, _ = draw(T * 1000 + d, T, d, dt)
        if not with_res:
            res = None
        gx, gres, gw = up(x, res, w)
        o = D.dora_rmsnorm(gx, gw, 1e-5, residual=gres, want_h=True, want_rstd=True, quantize=True,
                           group=group)
        h = R.norm_h(x, res)
        assert torch.equal(o["h"].cpu(), h)
        y, rstd = R.norm(h, w, 1e-5)
        E = (d / 64 + 64) * U
        within(o["rstd"], rstd, rstd * (E + 3 * U), "rstd")
        Ey = E + 6 * U
        within(o["y"], y, y.abs() * (Ey + half(dt)), "y")
        s_ref = R.quantize(y, group)[1].double()
        within(o["scale"], s_ref, s_ref * (Ey + 2 * U), "scale")
        s = R.spread(o["scale"].cpu(), d, group)
        within(o["q"].cpu().double() * s, y, s / 2 + y.abs() * Ey, "q scale")


@pytest.mark.parametrize("dt", [BF, F32])
def test_rmsnorm_single_outputs_agree_with_all_at_once(dt):
    x, res, w, _, _ = up(*draw(3, 11, 1000, dt))
    full = D.dora_rmsnorm(x, w, 1e-6, residual=res, want_rstd=True, quantize=True, group=64)
    say("rmsnorm y alone")
    assert torch.equal(D.dora_rmsnorm(x, w, 1e-6, residual=res, want_h=False)["y"], full["y"])
    say("rmsnorm 8 bits alone")
    o = D.dora_rmsnorm(x, w, 1e-6, residual=res, want_y=False, want_h=False, quantize=True, group=64)
    assert torch.equal(o["q"], full["q"]) and torch.equal(o["scale"], full["scale"])
    say("rmsnorm in place: h over the residual, y over x")
    x2, r2 = x.clone(), res.clone()
    out = {"y": x2, "h": r2, "rstd": torch.empty(11, device=DEV)}
    D.dora_rmsnorm(x2, w, 1e-6, residual=r2, out=out)
    assert torch.equal(x2, full["y"]) and torch.equal(r2, full["h"])
    say("rmsnorm in place: h over x")
    x3 = x.clone()
    D.dora_rmsnorm(x3, w, 1e-6, residual=res, out={"y": torch.empty_like(x), "h": x3})
    assert torch.equal(x3, full["h"])


@pytest.mark.parametrize("d", [1000, 40000])
def test_rmsnorm_in_place_over_long_rows(d):
    x, res, w, _, _ = up(*draw(4, 3, d, BF))
    full = D.dora_rmsnorm(x, w, 1e-6, residual=res, quantize=True, group=0)
    x2, r2 = x.clone(), res.clone()
    out = {"y": x2, "h": r2, "q": torch.empty_like(full["q"]), "scale": torch.empty_like(full["scale"])}
    say("rmsnorm in place", d)
    D.dora_rmsnorm(x2, w, 1e-6, residual=r2, out=out)
    assert torch.equal(x2, full["y"]) and torch.equal(r2, full["h"])
    assert torch.equal(out["q"], full["q"]) and torch.equal(out["scale"], full["scale"])


def test_rmsnorm_zero_and_nonfinite_rows():
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(1))
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 299] = float("nan")
    x[4, 0] = -float("inf")
    w = torch.ones(300)
    say("rmsnorm nonfinite rows")
    o = D.dora_rmsnorm(*up(x, w), 1e-6, quantize=True, want_rstd=True)
    y, s = o["y"].cpu(), o["scale"].cpu()[:, 0]
    assert (y[1] == 0).all() and s[1] == 0 and (o["q"][1] == 0).all()
    for t in (2, 3, 4):  # an infinity makes rstd 0 and its own y 0 * inf; a NaN makes all NaN
        assert torch.isnan(s[t]) and not torch.isfinite(y[t]).all()
    ref, _ = R.norm(x, w, 1e-6)
    for t in (0, 5):
        within(y[t:t + 1], ref[t:t + 1], ref[t:t + 1].abs() * 100 * U, "finite rows")
    assert torch.isfinite(s[[0, 5]]).all()


def test_rows_behind_the_last_are_left_alone():
    x, res, w, dy, dres = draw(9, 12, 200, BF)
    gx, gr, gw, gdy, gdr = up(x, res, w, dy, dres)
    big = {k: torch.full((12, 200), 7, dtype=t, device=DEV) for k, t in
           (("y", BF), ("h", BF), ("q", torch.int8), ("dx", BF))}
    rstd = torch.full((12,), 7.0, device=DEV)
    scale = torch.full((12, 1), 7.0, device=DEV)
    say("rmsnorm of 5 rows of 12")
    D.dora_rmsnorm(gx[:5], gw, residual=gr[:5],
                   out={"y": big["y"][:5], "h": big["h"][:5], "q": big["q"][:5], "rstd": rstd[:5],
                        "scale": scale[:5]})
    D.dora_rmsnorm_backward(gdy[:5], big["h"][:5], gw, rstd[:5], dres=gdr[:5],
                            out={"dx": big["dx"][:5], "dw": torch.empty(200, device=DEV)})
    torch.cuda.synchronize()
    for t in list(big.values()) + [rstd, scale]:
        assert (t[5:] == 7).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES + [(300, 136), (1000, 65), (70, 4096), (517, 2047),
                                           (9000, 40), (4100, 256), (2100, 1000)])
def test_rmsnorm_backward_matches_formula(T, d, dt):
    for with_dres in (True, False):
        say("rmsnorm backward", T, d, dt, with_dres)
        x, res, w, dy, dres = draw(T * 7 + d, T, d, dt)
        if not with_dres:
            dres = None
        gx, gres, gw, gdy, gdres = up(x, res, w, dy, dres)
        f = D.dora_rmsnorm(gx, gw, 1e-5, residual=gres, want_rstd=True)
        o = D.dora_rmsnorm_backward(gdy, f["h"], gw, f["rstd"], dres=gdres)
        h, rstd = f["h"].cpu(), f["rstd"].cpu()
        dx, dw, dot, each = R.norm_grad(dy, h, w, rstd, dres)
        r = rstd.double()[:, None]
        terms = (w.double() * dy.double()).abs() * r
        if with_dres:
            terms = terms + dres.double().abs()
        bound = (dx.abs() * half(dt) + 8 * U * terms
                 + h.double().abs() * r ** 3 / d * dot * ((d / 64 + 64) * U + 8 * U))
        within(o["dx"], dx, bound * (1 + 1e-6), "dx")
        within(o["dw"], dw, (T + 8) * U * each, "dw")


def test_rmsnorm_backward_matches_differences():
    """The fp32 kernel against central differences of the fp64 forward."""
    T, d, eps = 4, 37, 1e-4
    x, res, w, dy, dres = draw(21, T, d, F32)
    f = D.dora_rmsnorm(*up(x, w), eps, residual=res.to(DEV), want_rstd=True)
    say("rmsnorm backward against differences")
    o = D.dora_rmsnorm_backward(dy.to(DEV), f["h"], w.to(DEV), f["rstd"], dres=dres.to(DEV))
    h = f["h"].cpu().double()

    def loss(h, w):
        return float((R.norm(h, w, eps)[0] * dy.double()).sum() + (h * dres.double()).sum())

    step = 1e-5  # central differences: truncation step^2, rounding 2^-52 |loss| / step: 1e-8
    for t, j in [(0, 0), (1, 12), (2, 36), (3, 5), (0, 20)]:
        e = torch.zeros_like(h)
        e[t, j] = step
        diff = (loss(h + e, w.double()) - loss(h - e, w.double())) / (2 * step)
        assert abs(diff - float(o["dx"][t, j])) <= 1e-6 + 300 * U * (1 + abs(diff))
    for j in (0, 12, 36):
        e = torch.zeros(d, dtype=torch.float64)
        e[j] = step
        diff = (loss(h, w.double() + e) - loss(h, w.double() - e)) / (2 * step)
        assert abs(diff - float(o["dw"][j])) <= 1e-6 + 300 * U * (1 + abs(diff))


def test_rmsnorm_backward_in_place_over_dres_and_empty():
    x, res, w, dy, dres = up(*draw(8, 40, 520, BF))
    f = D.dora_rmsnorm(x, w, residual=res, want_rstd=True)
    a = D.dora_rmsnorm_backward(dy, f["h"], w, f["rstd"], dres=dres)
    keep = dres.clone()
    say("rmsnorm backward over dres")
    b = D.dora_rmsnorm_backward(dy, f["h"], w, f["rstd"], dres=keep,
                                out={"dx": keep, "dw": torch.empty(520, device=DEV)})
    assert torch.equal(a["dx"], keep) and torch.equal(a["dw"], b["dw"])
    say("rmsnorm T=0")
    e = torch.empty(0, 520, dtype=BF, device=DEV)
    f = D.dora_rmsnorm(e, w, residual=e, want_rstd=True, quantize=True, group=32)
    assert f["y"].shape == (0, 520) and f["scale"].shape == (0, 17)
    o = D.dora_rmsnorm_backward(e, e, w, f["rstd"])
    assert (o["dw"] == 0).all() and o["dx"].shape == (0, 520)


# ---------------------------------------------------------- rows to 8 bits
def special(T, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, 1, generator=g) * 3)
    return x.to(dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES + [(0, 64), (1000, 96)])
def test_quantize_gives_the_same_integers_and_scales(T, d, dt):
    x = special(T, d, dt, T + d)
    gx = x.to(DEV)
    for group in (0, 32, 64, 128, 256, 512):
        say("quantize", T, d, dt, group)
        q, s = D.dora_quantize_rows(gx, group=group)
        rq, rs = R.quantize(x, group)
        assert torch.equal(s.cpu(), rs), f"scales, group {group}"
        assert torch.equal(q.cpu(), rq), f"{int((q.cpu() != rq).sum())} integers, group {group}"
        for out in (BF, F32):
            say("dequantize", T, d, out, group)
            v = D.dora_dequantize_rows(q, s, group=group, dtype=out).cpu()
            want = (rq.float() * R.spread(rs, d, group).float()).to(out)
            assert torch.equal(v, want)


def test_quantize_ties_go_to_even():
    # scale exactly 1 and 2^-3: every half is a tie
    k = torch.arange(-126, 127).float()
    row = torch.cat([torch.tensor([127.0]), k + 0.5, k])
    x = torch.stack([row, row / 8, -row * 4])
    say("quantize ties")
    q, s = D.dora_quantize_rows(x.to(DEV))
    rq, rs = R.quantize(x, 0)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    assert q[0, 1 + 126] == 0 and q[0, 1 + 127] == 2  # 0.5 to 0 and 1.5 to 2


def test_quantize_near_ties_are_decided_exactly():
    # v = the two fp32 numbers around (k + 1/2) s for many scales
    g = torch.Generator().manual_seed(2)
    top = torch.rand(64, 1, generator=g) * 100 + 1
    s = (top.double() / 127).float().double()
    k = torch.arange(0, 126).double()[None] + 0.5
    tie = (k * s).float()
    x = torch.cat([top, tie, torch.nextafter(tie, torch.tensor(1e9)),
                   torch.nextafter(tie, torch.tensor(-1e9)), -tie], dim=1)
    say("quantize near ties")
    q, sc = D.dora_quantize_rows(x.to(DEV))
    rq, rs = R.quantize(x, 0)
    assert torch.equal(sc.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_quantize_extremes():
    big = torch.finfo(torch.float32).max
    tiny = 2.0 ** -149
    x = torch.randn(9, 256, generator=torch.Generator().manual_seed(3))
    x[0] = 0
    x[1] = big
    x[1, 1::2] = -big / 3
    x[2] = tiny
    x[3] = torch.arange(256) * tiny
    x[4] *= 2.0 ** -126
    x[5, 9] = float("inf")
    x[6, 200] = float("nan")
    x[7, 130] = -float("inf")
    gx = x.to(DEV)
    for group in (0, 128):
        say("quantize extremes", group)
        q, s = D.dora_quantize_rows(gx, group=group)
        rq, rs = R.quantize(x, group)
        assert torch.equal(torch.isnan(s.cpu()), torch.isnan(rs))
        assert torch.equal(torch.nan_to_num(s.cpu()), torch.nan_to_num(rs))
        assert torch.equal(q.cpu(), rq)
        v = D.dora_dequantize_rows(q, s, group=group, dtype=F32).cpu()
        assert (v[0] == 0).all() and torch.isfinite(v[1]).all()
        assert torch.isnan(v[5, 9]) and torch.isnan(v[6, 200]) and torch.isnan(v[7, 130])
        assert torch.isfinite(v[5, 200]).all() == (group == 128)


def test_rows_calls_refuse_what_they_cannot_read():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    bad = [lambda: D.dora_rmsnorm(x.T, w), lambda: D.dora_rmsnorm(x, w[:32]),
           lambda: D.dora_rmsnorm(x, w, residual=x[:2]), lambda: D.dora_rmsnorm(x, w, group=48),
           lambda: D.dora_rmsnorm(x, w, want_y=False), lambda: D.dora_rmsnorm(x[None], w),
           lambda: D.dora_rmsnorm(x, w, out={"y": x.clone(), "q": torch.empty(4, 64, dtype=torch.int8, device=DEV)}),
           lambda: D.dora_rmsnorm(x, w, out={"z": x}), lambda: D.dora_quantize_rows(x.T),
           lambda: D.dora_quantize_rows(x, group=7),
           lambda: D.dora_dequantize_rows(torch.zeros(4, 64, dtype=torch.int8, device=DEV), w[:4]),
           lambda: D.dora_rmsnorm_backward(x, x, w, w[:3])]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(k)
    for call in (lambda: D.dora_rmsnorm(x.half(), w.half()), lambda: D.dora_rmsnorm(x, w.bfloat16()),
                 lambda: D.dora_dequantize_rows(x, w[:4, None])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(D.DoraError):
        D.dora_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(D.DoraError):
        D.dora_rmsnorm(x, w, out={"y": x, "h": x})


# ------------------------------------------------------------ the largest sizes
def test_more_rows_than_one_launch_holds():
    """70 million rows of 4: a workgroup a row would be more threads than a
    launch takes."""
    T, d = 70_000_000, 4
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(T, d, generator=g, device=DEV, dtype=BF)
    say("quantize", T, d)
    q, s = D.dora_quantize_rows(x)
    at = torch.tensor([0, 1, 2 ** 20 - 1, 2 ** 20, 67_108_863, 67_108_864, T - 2, T - 1])
    rq, rs = R.quantize(x[at.to(DEV)].cpu(), 0)
    assert torch.equal(q[at.to(DEV)].cpu(), rq) and torch.equal(s[at.to(DEV)].cpu(), rs)
    say("dequantize", T, d)
    v = D.dora_dequantize_rows(q, s)
    assert torch.equal(v[at.to(DEV)].cpu(), (rq.float() * rs).to(BF))
    del q, s, v
    w = torch.ones(d, device=DEV, dtype=BF)
    say("rmsnorm", T, d)
    o = D.dora_rmsnorm(x, w, 1e-5)
    ref, _ = R.norm(x[at.to(DEV)].cpu(), w.cpu(), 1e-5)
    within(o["y"][at.to(DEV)], ref, ref.abs() * (2.0 ** -8 + 100 * U), "y")


def test_offsets_past_32_bits():
    T, d = 1_050_000, 2056   # 2.16e9 elements
    g = torch.Generator(DEV).manual_seed(2)
    x = torch.randn(T, d, generator=g, device=DEV, dtype=BF)
    at = torch.tensor([0, T // 2, 1_044_494, 1_044_495, T - 1])
    for group in (0, 128):
        say("quantize", T, d, group)
        q, s = D.dora_quantize_rows(x, group=group)
        rq, rs = R.quantize(x[at.to(DEV)].cpu(), group)
        assert torch.equal(q[at.to(DEV)].cpu(), rq) and torch.equal(s[at.to(DEV)].cpu(), rs)
        say("dequantize", T, d, group)
        v = D.dora_dequantize_rows(q, s, group=group)
        assert torch.equal(v[at.to(DEV)].cpu(), (rq.float() * R.spread(rs, d, group).float()).to(BF))
        del q, s, v
    w = (1 + torch.randn(d, generator=g, device=DEV) / 8).to(BF)
    say("rmsnorm and its gradient", T, d)
    f = D.dora_rmsnorm(x, w, 1e-5, want_rstd=True)
    o = D.dora_rmsnorm_backward(f["y"], x, w, f["rstd"])
    xs, ys = x[at.to(DEV)].cpu(), f["y"][at.to(DEV)].cpu()
    ref, _ = R.norm(xs, w.cpu(), 1e-5)
    within(ys, ref, ref.abs() * (2.0 ** -8 + (d / 64 + 64) * U), "y")
    rs = f["rstd"][at.to(DEV)].cpu()
    dx, _, dot, _ = R.norm_grad(ys, xs, w.cpu(), rs, None)
    r = rs.double()[:, None]
    bound = (dx.abs() * 2.0 ** -8 + 8 * U * (w.cpu().double() * ys.double()).abs() * r
             + xs.double().abs() * r ** 3 / d * dot * ((d / 64 + 64) * U + 8 * U))
    within(o["dx"][at.to(DEV)], dx, bound * (1 + 1e-6), "dx")
    # dw of one column in 64 bits: at most T / 1 terms summed by parts of T / parts
    col = (f["y"][:, 5].double() * x[:, 5].double() * f["rstd"].double())
    assert abs(float(o["dw"][5]) - float(col.sum())) <= (T / 256 + 300) * U * float(col.abs().sum())


def test_long_rows():
    for T, d in ((1, 3_000_001), (3, 600_000)):
        x, res, w, dy, dres = draw(d, T, d, BF)
        gx, gres, gw, gdy, gdres = up(x, res, w, dy, dres)
        say("rmsnorm", T, d)
        f = D.dora_rmsnorm(gx, gw, 1e-5, residual=gres, want_rstd=True, quantize=True, group=256)
        h = R.norm_h(x, res)
        y, _ = R.norm(h, w, 1e-5)
        E = (d / 64 + 70) * U
        within(f["y"], y, y.abs() * (E + 2.0 ** -8), "y")
        s = R.spread(f["scale"].cpu(), d, 256)
        within(f["q"].cpu().double() * s, y, s / 2 + y.abs() * E, "q scale")
        say("rmsnorm backward", T, d)
        o = D.dora_rmsnorm_backward(gdy, f["h"], gw, f["rstd"], dres=gdres)
        dx, dw, dot, each = R.norm_grad(dy, h, w, f["rstd"].cpu(), dres)
        within(o["dw"], dw, (T + 8) * U * each, "dw")
        r = f["rstd"].cpu().double()[:, None]
        bound = (dx.abs() * 2.0 ** -8
                 + 8 * U * ((w.double() * dy.double()).abs() * r + dres.double().abs())
                 + h.double().abs() * r ** 3 / d * dot * E)
        within(o["dx"], dx, bound * (1 + 1e-6), "dx")
