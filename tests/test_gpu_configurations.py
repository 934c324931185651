"""GPU: every kernel configuration of the int8 product and of the bf16 product of any
width, each at a size that reaches it (the launched kernel's name says so), at ragged
and whole edges, in both output types, over more rows of tiles than one.

int8: the sums are exact, tolerances as in test_gpu_linear_quantized.  bf16: values
-1, 0, 1, so that every sum is exact in fp32 and each result is the exact one rounded
once."""
import pytest
import torch

import rows8_ref as R
from dora_adapter_amd import dora as D
from gpu_util import say
from test_gpu_persistent import _kernels

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

DMA, ANY8 = "gemm_i8_dma_kernel<", "gemm_i8_general_kernel<"
# (tokens, d_in, d_out, kernel, sums split over K).  Pipelined tiles: once with fewer
# and once with more items than workgroups, d_out of whole 16-byte chunks of y and not.
INT8 = [
    (411, 1024, 24902, DMA + "256, 256,", False),
    (1947, 928, 12456, DMA + "256, 256,", False),
    (133, 7568, 16607, DMA + "256, 256,", True),
    (131, 6816, 17256, DMA + "256, 256,", True),
    (1213, 208, 18623, DMA + "128, 128, 2, 2, 2,", False),
    (411, 304, 24776, DMA + "128, 128, 2, 2, 2,", False),
    (139, 9408, 5466, DMA + "128, 128, 2, 2, 2,", True),
    (139, 9408, 5464, DMA + "128, 128, 2, 2, 2,", True),
    (3419, 448, 1114, DMA + "128, 128, 2, 2, 4,", False),
    (1100, 1040, 17000, DMA + "128, 128, 2, 2, 4,", False),
    (66, 11600, 2430, DMA + "128, 128, 2, 2, 4,", True),
    (66, 11600, 2432, DMA + "128, 128, 2, 2, 4,", True),
    (6781, 416, 167, DMA + "128, 64,", False),
    (8316, 320, 392, DMA + "128, 64,", False),
    (2407, 4064, 18, DMA + "128, 64,", True),
    (2407, 4064, 16, DMA + "128, 64,", True),
    (135, 336, 17597, DMA + "64, 64,", False),
    (1238, 96, 176, DMA + "64, 64,", False),
    (554, 13408, 25, DMA + "64, 64,", True),
    (554, 13408, 24, DMA + "64, 64,", True),
    (1, 640, 520, "gemm_i8_rows_kernel<1, 16,", False),
    (16, 400, 12001, "gemm_i8_rows_kernel<1, 32,", False),
    (17, 1552, 4096, "gemm_i8_rows_kernel<2, 16,", False),
    (32, 272, 4099, "gemm_i8_rows_kernel<2, 64,", False),
    (33, 1040, 2049, "gemm_i8_rows_kernel<4, 16,", False),
    (64, 144, 8191, "gemm_i8_rows_kernel<4, 32,", False),
    (5, 1, 7, ANY8 + "64, 2, 1, true,", False),
    (300, 1029, 260, ANY8 + "64, 2, 3,", True),
    (777, 133, 411, ANY8 + "64, 2, 3,", False),
    (2050, 1030, 4099, ANY8 + "128, 2, 2,", False),
    (2049, 131, 4104, ANY8 + "128, 2, 2,", False),
    (2048, 1029, 2047, ANY8 + "128, 2, 2,", True),
    (4100, 130, 4100, ANY8 + "256, 4, 1,", False),
    (4099, 1031, 4101, ANY8 + "256, 4, 1,", False),
]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d_in,d_out,kernel,split", INT8)
def test_int8_configuration(T, d_in, d_out, kernel, split, dt):
    g = torch.Generator().manual_seed(T + d_out)
    xq = torch.randint(-128, 128, (T, d_in), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (d_out, d_in), generator=g, dtype=torch.int8)
    xs = torch.rand(T, 1, generator=g) * 0.1 + 0.01
    ws = torch.rand(d_out, 1, generator=g) * 0.01 + 0.001
    dev = [t.to(DEV) for t in (xq, xs, wq, ws)]
    say("int8 linear", T, d_in, d_out, dt, kernel)
    y = torch.full((T + 3, d_out), 7.0, dtype=dt, device=DEV)
    D.dora_linear_quantized(*dev, y=y[:T])
    ref = R.linear(xq, xs, wq, ws)
    off = (y[:T].cpu().double() - ref).abs()
    lim = ref.abs() * (3.1 * 2.0 ** -24 + torch.finfo(dt).eps / 2)
    assert (off <= lim).all(), f"{int((off > lim).sum())} of {off.numel()} off"
    assert (y[T:] == 7).all()
    names = _kernels(lambda: D.dora_linear_quantized(*dev, y=y[:T]))
    assert any(kernel in k for k in names), names
    assert any("i8_finish_kernel" in k for k in names) == split, names


ANY = "gemm_bf16_any_kernel<%d, "


def ints(g, *shape, p=1.0):
    v = torch.randint(-1, 2, shape, generator=g)
    return (v * (torch.rand(shape, generator=g) < p)).double()


# (T, d_in, d_out, r): widths of no multiple; 128 x 128 tiles store x W^T, dx, dA or dB
WIDE = [(2049, 2051, 2053, 37), (300, 2051, 2053, 2050), (4100, 70, 8191, 3), (8193, 1027, 515, 5)]


@pytest.mark.parametrize("T,d_in,d_out,r", WIDE)
def test_bf16_any_width_128_tiles(T, d_in, d_out, r):
    """The gradients' and x W^T's storing products on 128 x 128 tiles in all three
    layouts, dx over two K segments of which the first ends inside a step."""
    g = torch.Generator().manual_seed(T + r)
    dy, W, A, B, P = (ints(g, T, d_out, p=0.05), ints(g, d_out, d_in), ints(g, r, d_in),
                      ints(g, d_out, r), ints(g, T, r))
    x, y = ints(g, T, d_in), ints(g, T, d_out)
    one = torch.ones(d_out, device=DEV)
    dev = [t.to(BF).to(DEV) for t in (dy, x, W, A, B, P, y)]
    gdy, gx, gW, gA, gB, gP, gy = dev
    Q = dy @ B
    assert Q.abs().max() <= 256  # exact in bf16
    want = {"dx": dy @ W + Q @ A, "dA": Q.T @ x, "dB": dy.T @ P, "dm": (dy * y).sum(0)}
    say("backward on integers", T, d_in, d_out, r)
    got = D.dora_backward(gdy, gx, gW, gA, gB, one, one, 1.0, gP, gy)
    for k, v in want.items():
        assert torch.equal(got[k].cpu(), v.to(got[k].dtype)), k
    say("linear on integers", T, d_in, d_out)
    assert torch.equal(D.dora_linear(gx, gW).cpu(), (x @ W.T).to(BF))


def test_bf16_any_width_128_tiles_are_reached():
    """Between them the sizes above store on 128 x 128 tiles in each layout."""
    seen = set()
    for T, d_in, d_out, r in WIDE:
        z = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
        one = torch.ones(d_out, device=DEV)
        say("kernels of the backward", T, d_in, d_out, r)
        ops = (z(T, d_out), z(T, d_in), z(d_out, d_in), z(r, d_in), z(d_out, r))
        names = _kernels(lambda: D.dora_backward(*ops, one, one, 1.0, z(T, r), z(T, d_out)))
        names += _kernels(lambda: D.dora_linear(ops[1], ops[2]))
        seen |= {k.split("gemm_bf16_any_kernel<")[1].split(">")[0] for k in names
                 if ANY % 128 in k}
    for layout in ("true, true, false", "true, false, false", "false, false, false"):
        assert any(k.endswith(layout) for k in seen), (layout, seen)
