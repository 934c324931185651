"""GPU: the int8 linear layer over the whole range of fp32 scales.

The sum's conversion, its products with the two scales and the output's rounding
are relative to y (4 u, u = 2^-24) wherever y itself is a normal number, however
small or large either scale is: powers of two move no bit, so the bound is that of
ordinary scales."""
import pytest
import torch

import rows8_ref as R
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32

# one size for each kernel that scales sums: a few tokens; 64 x 64, 128 x 128 and
# 256 x 256 tiles of any width; pipelined tiles with the scales in registers and
# in LDS; split sums, pipelined and of any width
SIZES = [(3, 512, 40), (40, 513, 37), (2050, 70, 4099), (4100, 70, 4100), (100, 512, 9000),
         (411, 1024, 24902), (96, 8192, 64), (300, 4099, 260)]


def operands(T, d_in, d_out):
    g = torch.Generator().manual_seed(T + d_in + d_out)
    xq = torch.randint(-127, 128, (T, d_in), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (d_out, d_in), generator=g, dtype=torch.int8)
    xq[0] = 0
    xs, ws = (torch.rand(n, 1, generator=g).double() + 1 for n in (T, d_out))
    return xq, xs, wq, ws


@pytest.mark.parametrize("T,d_in,d_out", SIZES)
def test_any_scale_whose_result_is_a_number(T, d_in, d_out):
    xq, xs, wq, ws = operands(T, d_in, d_out)
    dev = [t.to(DEV) for t in (xq, wq)]
    sums = xq.double() @ wq.double().T
    # exponents of the scales; the result's stays within 2^-100 .. 2^90
    for ex, ew in ((-126, 100), (-126, 121), (-118, 118), (-110, 90), (-103, 60), (-140, 120),
                   (60, -126), (95, -60), (96, -80), (97, -100), (110, -110), (120, -126),
                   (121, -140), (126, -60), (104, -104), (-20, 105)):
        sx, sw = (xs * 2.0 ** ex).float(), (ws * 2.0 ** ew).float()
        say("int8 linear, scales of 2^%d and 2^%d" % (ex, ew), T, d_in, d_out)
        y = D.dora_linear_quantized(dev[0], sx.to(DEV), dev[1], sw.to(DEV), dtype=F32).cpu()
        ref = sums * sx.double() * sw.double().T
        off = (y.double() - ref).abs()
        assert (off <= ref.abs() * 4.1 * 2.0 ** -24).all(), (
            f"scales of 2^{ex} and 2^{ew}: worst {float((off / ref.abs()).nan_to_num().max()):.2e}")


@pytest.mark.parametrize("T,d_in,d_out", SIZES)
def test_overflow_zero_and_nonfinite_scales(T, d_in, d_out):
    xq, xs, wq, ws = operands(T, d_in, d_out)
    big, w_big = (xs * 2.0 ** 126).float(), (ws * 2.0 ** 126).float()
    big[1], big[2] = float("nan"), float("inf")
    say("int8 linear, scales whose product overflows", T, d_in, d_out)
    y = D.dora_linear_quantized(*[t.to(DEV) for t in (xq, big, wq, w_big)], dtype=F32).cpu()
    sums = xq.double() @ wq.double().T
    assert (y[0] == 0).all() and torch.isnan(y[1]).all()
    rows = [t for t in range(min(T, 200)) if t not in (0, 1)]
    want = torch.sign(sums[rows]) * float("inf")
    want[0][sums[2] == 0] = float("nan")  # 0 times an infinite scale
    if T > 3:
        want[1:][sums[rows[1:]] == 0] = 0.0
    assert torch.equal(torch.isnan(want), torch.isnan(y[rows].double()))
    assert torch.equal(want.nan_to_num(0.0, 1.0, -1.0), y[rows].double().nan_to_num(0.0, 1.0, -1.0))


def test_rows_as_the_quantiser_makes_them():
    """The smallest and largest scales that the quantiser hands out."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 256, generator=g) * 2.0 ** torch.tensor([-124., -118, -110, 0, 112, 118])[:, None]
    w = torch.randn(48, 256, generator=g)
    xq, xs = D.dora_quantize_rows(x.to(DEV))
    wq, ws = D.dora_quantize_rows(w.to(DEV))
    say("int8 linear, rows near the ends of fp32's range")
    y = D.dora_linear_quantized(xq, xs, wq, ws, dtype=F32).cpu()
    ref = R.linear(xq.cpu(), xs.cpu(), wq.cpu(), ws.cpu())
    # (2^-150: half of the smallest denormal step, where y is one)
    assert ((y.double() - ref).abs() <= ref.abs() * 4.1 * 2.0 ** -24 + 2.0 ** -149).all()
