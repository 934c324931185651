"""GPU: the norm and its gradient over fp32's range of magnitudes.

A row of any magnitude for which rstd is a number has the same relative errors as a
row of unit magnitude: the bounds are those of test_gpu_rows8 (u = 2^-24; sums of at
most d / 64 + 64 terms in a chain), with one step of the smallest denormal more for
every rounding that meets one."""
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


def within(got, ref, bound, what):
    got = got.cpu().double()
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert (off <= bound).all(), (f"{what}: {int((off > bound).sum())} of {off.numel()} off, worst "
                                  f"{float((off / bound.clamp_min(1e-300)).max()):.2f}x the bound")


# widths of every form of the kernels (a workgroup's registers, one to four vectors a
# thread, and longer rows) and enough rows for the form of many rows
SHAPES = [(5, 33), (600, 136), (3, 2048), (520, 4100), (2, 16384), (2, 28672), (3, 40000)]


def rows(T, d, e, dt, seed):
    g = torch.Generator().manual_seed(seed)
    h, dy, dres = (torch.randn(T, d, generator=g) for _ in range(3))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dt)
    # a row in three stays at unit magnitude
    scale = torch.full((T, 1), 2.0 ** e)
    scale[1::3] = 1.0
    return (h * scale).to(dt), w, dy, dres, scale


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rmsnorm_of_small_and_large_rows(T, d, dt):
    for e, eps in ((-100, 0.0), (-72, 0.0), (-65, 0.0), (-52, 0.0), (-60, 2.0 ** -118), (55, 1e-6),
                   (62, 1e-6), (64, 0.0), (80, 1e-6), (100, 1e-6), (118, 1e30)):
        h, w, _, _, _ = rows(T, d, e, dt, T + d)
        say("rmsnorm", T, d, dt, "rows of 2^%d" % e)
        o = D.dora_rmsnorm(h.to(DEV), w.to(DEV), eps, want_rstd=True, quantize=True)
        y, rstd = R.norm(h, w, float(torch.tensor(eps)))
        E = (d / 64 + 64) * U
        within(o["rstd"], rstd, rstd * (E + 6 * U), f"rstd, 2^{e}")
        Ey = E + 9 * U
        within(o["y"], y, y.abs() * (Ey + half(dt)) + 2.0 ** -133, f"y, 2^{e}")
        s = o["scale"].cpu().double()
        within(o["q"].cpu().double() * s, y, s / 2 + y.abs() * Ey + 2.0 ** -126, f"q scale, 2^{e}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rmsnorm_gradient_of_small_and_large_rows(T, d, dt):
    """dx and dw from h of 2^e and dy of 2^f: sums whose terms leave fp32's range
    before they meet rstd, coefficients that leave it before they meet h."""
    for e, f in ((-100, 0), (-65, 0), (-65, 40), (-65, -100), (0, 100), (64, 60), (100, 60), (100, 0),
                 (40, -100), (-40, 80)):
        h, w, dy, dres, scale = rows(T, d, e, dt, T + d)
        dy = (dy * 2.0 ** f).to(dt)
        rstd = R.norm(h, w, 0.0)[1].float()
        # the stream's gradient, of dx's own magnitude
        dres = (dres * 2.0 ** f / scale).to(dt)
        for res in (None, dres):
            say("rmsnorm backward", T, d, dt, "h of 2^%d, dy of 2^%d" % (e, f), res is not None)
            o = D.dora_rmsnorm_backward(*[t.to(DEV) for t in (dy, h, w, rstd)],
                                        dres=None if res is None else res.to(DEV))
            dx, dw, dot, each = R.norm_grad(dy, h, w, rstd, res)
            r = rstd.double()[:, None]
            terms = (w.double() * dy.double()).abs() * r
            if res is not None:
                terms = terms + res.double().abs()
            bound = (dx.abs() * half(dt) + 8 * U * terms
                     + h.double().abs() * r ** 3 / d * dot * ((d / 64 + 64) * U + 8 * U))
            tiny = 2.0 ** -133 if dt == BF else 2.0 ** -148
            # (a term's own denormal step meets rstd: of rows of 2^e, 2^-e of it)
            within(o["dx"], dx, bound * (1 + 1e-6) + tiny + 2.0 ** -148 * r, f"dx, 2^{e}, 2^{f}")
            within(o["dw"], dw, (T + 8) * U * each + T * 2.0 ** -148, f"dw, 2^{e}, 2^{f}")


def test_zero_rows_and_infinities_as_before():
    x = torch.zeros(4, 300)
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = 3.0e38
    say("rmsnorm, a row of zeros, an infinity, a NaN, the largest values")
    o = D.dora_rmsnorm(x.to(DEV), torch.ones(300, device=DEV), 1e-6, want_rstd=True)
    y, rstd = o["y"].cpu(), o["rstd"].cpu()
    assert (y[0] == 0).all() and abs(float(rstd[0]) - 1e3) < 1e-2
    assert float(rstd[1]) == 0 and torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()
    assert torch.isnan(y[2]).all()
    # (rstd is a denormal number of 21 bits there)
    assert ((y[3] - 1).abs() <= 2.0 ** -20).all()
