"""GPU: rows to 4 bits and back, and the linear layer from them, against their
plain forms in 64 bits.

Rows: the same values and scales, exactly (the rounding is decided exactly, and
a scale of six bits times a code of two is a bf16 number).
The linear layer (u = 2^-24): up to 256 tokens exact products and fp32 sums in
any order, d_in terms, each group's sum times its scale: (d_in + 8) u sum |x w|
at most (no order of d_in additions is off by more), and the output's rounding,
2^-8 |y| for bf16 and 2^-24 |y| for fp32; more tokens the same bound, the
weights being exact."""
import pytest
import torch

import around_ref as R
from around_ref import U, half
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def same(got, ref, what):
    got = got.cpu().double()
    assert got.shape == ref.shape, what
    assert torch.equal(got.isnan(), ref.isnan()), what
    bad = (got != ref) & ~ref.isnan()
    assert not bad.any(), f"{what}: {int(bad.sum())} differ, first {got[bad][:3]} for {ref[bad][:3]}"


def check_rows(x, group):
    T, d = x.shape
    say("to 4 bits", T, d, x.dtype, group)
    codes, scale = D.dora_quantize_fourbit(x.to(DEV), group=group)
    values, s = R.fourbit(x, group)
    same(scale, s, "scale")
    c = codes.cpu()
    full = R.unpack(c)
    ok = ~s.isnan().repeat_interleave(group, dim=1)
    assert torch.equal(full[:, :d][ok[:, :d]], values[ok[:, :d]])
    assert torch.count_nonzero(full[:, d:]) == 0
    for dt in (BF, F32):
        out = D.dora_dequantize_fourbit(codes, scale, d, group=group, dtype=dt)
        same(out, values * s.repeat_interleave(group, dim=1)[:, :d], f"restored {dt}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 32), (3, 33), (5, 100), (2, 512), (7, 513), (33, 1029),
                                 (3, 4096), (2, 8200), (300, 64), (1000, 31), (1, 40003)])
def test_rows(T, d, dt):
    g = torch.Generator().manual_seed(T * 1000 + d)
    for group in (32, 64, 128, 256, 512):
        x = torch.randn(T, d, generator=g) * torch.exp2(4 * torch.randn(T, 1, generator=g))
        check_rows(x.to(dt), group)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_at_every_tie_and_next_to_it(dt):
    """Every scale's significand, every border between two codes, and the numbers around it."""
    rows = []
    step = torch.finfo(dt).eps
    for k in range(32):
        s = (32 + k) / 32.0
        border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * s
        near = torch.cat([border, border * (1 + step), border * (1 - step), border * (1 + 3 * step),
                          border * (1 - 3 * step)])
        row = torch.zeros(128, dtype=torch.float64)
        row[:35], row[35:70], row[70] = near, -near, 6 * s
        rows.append(row)
    x = torch.stack(rows)
    for power in (-100, -3, 0, 50, 120):
        check_rows((x * 2.0 ** power).to(dt), 128)


@pytest.mark.parametrize("dt", [BF, F32])
def test_scales_at_every_tie_and_next_to_it(dt):
    """max / 6 halfway between two numbers of six bits, and next to that."""
    half_way = torch.tensor([(32 + k) / 32.0 + 1 / 64.0 for k in range(32)], dtype=torch.float64) * 6
    step = torch.finfo(dt).eps
    rows = torch.cat([half_way, half_way * (1 + step), half_way * (1 - step)])[:, None]
    x = torch.cat([rows, -rows / 3, rows / 7], dim=1)
    check_rows(x.to(dt), 32)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_zeros_tiny_huge_and_nonfinite_values(dt):
    big = torch.finfo(dt).max
    x = torch.randn(9, 200, generator=torch.Generator().manual_seed(4))
    x[0] = 0
    x[1, 64:128] = 0
    x[2] *= 2.0 ** -126
    x[3] = 2.0 ** -133
    x[4] = 2.0 ** -126 * torch.sign(x[4])
    x[5, 100] = big
    x[6, 150] = float("inf")
    x[7, 3] = float("nan")
    x[8, 199] = -float("inf")
    x = x.to(dt)
    check_rows(x, 64)
    x[5] = big
    check_rows(x, 32)


def test_rows_past_32_bit_offsets():
    rows, d = (1 << 32) // 8192 + 3, 8192
    say("to 4 bits past 2^32 elements")
    x = torch.randn(64, d, device=DEV, dtype=BF).repeat(rows // 64 + 1, 1)[:rows]
    codes, scale = D.dora_quantize_fourbit(x, group=32)
    tail = slice(rows - 2, rows)
    values, s = R.fourbit(x[tail].cpu(), 32)
    same(scale[tail], s, "scale")
    same(R.unpack(codes[tail].cpu()), values, "codes")
    out = D.dora_dequantize_fourbit(codes, scale, d, group=32, out=x)
    same(out[tail], values * s.repeat_interleave(32, dim=1), "restored")


def weight(seed, d_out, d_in, group, bits=6):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(d_out, d_in, generator=g) * d_in ** -0.5
    W[:: 7] *= 20.0
    codes, scale = D.dora_quantize_fourbit(W.to(DEV), group=group)
    if bits > 6:  # scales that are not the quantiser's
        scale = scale * (1 + 2.0 ** -7 * torch.randint(0, 4, scale.shape, generator=g).to(DEV))
        scale = scale.to(BF)
    return codes, scale


def check_linear(T, d_in, d_out, dt, group, bits=6, x=None):
    say("linear from 4 bits", T, d_in, d_out, dt, group, bits)
    codes, scale = weight(T + d_in, d_out, d_in, group, bits)
    if x is None:
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, d_in, generator=g)
        x[:, d_in // 3] *= 12
        x = x.to(dt)
    y = D.dora_linear_fourbit(x.to(DEV), codes, scale, group=group)
    W = R.restored(codes.cpu(), scale.cpu(), d_in, group)
    rounded = W if T <= 256 else W.to(dt).double()
    ref = x.double() @ rounded.T
    bound = (d_in + 8) * U * (x.double().abs() @ W.abs().T) + ref.abs() * half(dt)
    off = (y.cpu().double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (off <= bound).all(), f"worst {float((off / bound.clamp_min(1e-300)).max()):.2f}x the bound"
    return x, codes, scale, y


@pytest.mark.parametrize("group", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 16, 17, 33, 64])
def test_linear_few_tokens(T, group):
    check_linear(T, 1029, 515, BF, group)
    check_linear(T, 2048, 100, F32, group)
    check_linear(T, 777, 33, F32, group, bits=8)
    check_linear(T, 4096, 256, BF, group, bits=8)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d_in,d_out", [(1, 1), (7, 3), (31, 17), (32, 16), (33, 40), (255, 31),
                                        (256, 32), (257, 33), (288, 64), (511, 65), (1024, 7),
                                        (3000, 129), (8192, 48), (12290, 40), (40000, 16)])
def test_linear_sizes(d_in, d_out, dt):
    for T, group in ((1, 32), (3, 128), (9, 64), (40, 512), (64, 32)):
        check_linear(T, d_in, d_out, dt, group)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d_in,d_out,group", [
    (65, 1029, 515, 32), (100, 256, 1024, 64), (129, 100, 70, 128), (256, 300, 40, 64),
    (257, 1029, 515, 32), (300, 2048, 512, 128), (270, 513, 9, 512), (400, 31, 70, 32)])
def test_linear_more_tokens(T, d_in, d_out, group, dt):
    check_linear(T, d_in, d_out, dt, group)
    check_linear(T, d_in, d_out, dt, group, bits=8)


@pytest.mark.parametrize("dt,T,d_out", [
    (BF, 4, 30000), (BF, 16, 12400), (BF, 16, 4000), (BF, 40, 24700), (BF, 64, 12300), (BF, 20, 24600),
    (BF, 20, 12300), (BF, 20, 4000), (BF, 200, 6200), (F32, 16, 12400), (F32, 30, 4000),
    (F32, 4, 4200)])
def test_linear_every_kernel(dt, T, d_out):
    """Enough channels that each tile rule is met from both sides, tiles cut off at the end, and
    workgroups that walk several tiles."""
    for d_in, group in ((512, 128), (700, 32), (1500, 256)):
        check_linear(T, d_in, d_out - 3, dt, group)


@pytest.mark.parametrize("T", [4, 16, 17, 32, 33, 64, 100])
@pytest.mark.parametrize("d_out", [70, 4000, 12301, 24590])
def test_linear_groups_of_64(T, d_out):
    """Each tile rule again with four scales a line, the last line a whole one and not."""
    for d_in in (768, 1091):
        check_linear(T, d_in, d_out, BF, 64)


@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_in_panels(dt):
    """A weight of more rows than a panel holds: the last panel is a short one."""
    d_in = 1 << 17
    check_linear(258, d_in, 2 * (512 if dt == BF else 256) + 37, dt, 512)


def test_linear_nonfinite_tokens_and_scales():
    codes, scale = weight(3, 50, 600, 64)
    x = torch.randn(6, 600, generator=torch.Generator().manual_seed(8))
    x[1, 5], x[2, 599], x[3, 300] = float("inf"), float("nan"), -float("inf")
    W = R.restored(codes.cpu(), scale.cpu(), 600, 64)
    for dt in (BF, F32):
        for rows in (slice(0, 3), slice(0, 6)):
            say("non-finite tokens", dt, rows)
            xs = x[rows].to(dt)
            ref = xs.double() @ W.T
            y = D.dora_linear_fourbit(xs.to(DEV), codes, scale, group=64).cpu().double()
            assert torch.equal(y.isnan(), ref.isnan())
            inf = ref.isinf()
            assert torch.equal(y[inf], ref[inf])
            assert torch.equal(y.isfinite(), ref.isfinite())
    # a NaN in the lower bits alone
    bits = torch.full((1, 600), 0x3F800000, dtype=torch.int32)
    bits[0, 7] = 0x7F800001
    y = D.dora_linear_fourbit(bits.view(F32).to(DEV), codes, scale, group=64)
    assert y.isnan().all()
    scale[7, 2] = float("nan")
    y = D.dora_linear_fourbit(x[:1].to(BF).to(DEV), codes, scale, group=64)
    assert y[0, 7].isnan() and y[0, :7].isfinite().all() and y[0, 8:].isfinite().all()


@pytest.mark.parametrize("T", [1, 9, 40])
def test_linear_tokens_of_any_magnitude(T):
    """fp32 tokens down to 2^-95 and up to 2^100 keep 24 bits."""
    g = torch.Generator().manual_seed(11)
    for power in (-95, 100):
        x = torch.randn(T, 700, generator=g).clamp(-8, 8)
        x = torch.sign(x) * x.abs().clamp_min(2.0 ** -5) * 2.0 ** power
        check_linear(T, 700, 64, F32, 128, x=x)


def test_linear_past_32_bit_offsets():
    """A weight of over 2^32 bytes of codes: its last channels."""
    d_in, d_out = 8192, (1 << 32) // 4096 + 20
    say("linear from 4 bits past 2^32 bytes of codes")
    codes = torch.randint(0, 256, (1024, d_in // 2), device=DEV, dtype=torch.uint8)
    codes = codes.repeat(d_out // 1024 + 1, 1)[:d_out]
    scale = torch.rand(1024, d_in // 32, device=DEV).to(BF).repeat(d_out // 1024 + 1, 1)[:d_out]
    x = torch.randn(20, d_in, device=DEV, dtype=BF)
    for T in (1, 20):
        y = D.dora_linear_fourbit(x[:T].contiguous(), codes, scale, group=32)
        ref = D.dora_linear_fourbit(x[:T].contiguous(), codes[-40:].contiguous(),
                                    scale[-40:].contiguous(), group=32)
        W = R.restored(codes[-40:].cpu(), scale[-40:].cpu(), d_in, 32)
        full = x[:T].cpu().double() @ W.T
        bound = (d_in + 8) * U * (x[:T].cpu().double().abs() @ W.abs().T) + full.abs() * half(BF)
        for got in (y[:, -40:], ref):
            assert ((got.cpu().double() - full).abs() <= bound).all()


def test_linear_no_tokens_and_padding():
    codes, scale = weight(1, 40, 100, 32)
    assert D.dora_linear_fourbit(torch.empty(0, 100, device=DEV, dtype=BF), codes, scale,
                                 group=32).shape == (0, 40)
    # what lies past the last column is no part of the matrix
    x = torch.randn(3, 100, device=DEV, dtype=BF)
    y = D.dora_linear_fourbit(x, codes, scale, group=32)
    codes[:, 50:] = 0x5A
    assert torch.equal(D.dora_linear_fourbit(x, codes, scale, group=32), y)


@pytest.mark.parametrize("T", [1, 20, 200, 300])
def test_streams_and_graphs(T):
    x, codes, scale, y = check_linear(T, 1024, 640, BF, 128)
    x = x.to(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(D.dora_linear_fourbit(x, codes, scale))
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)
    need = D.dora_linear_fourbit_workspace(T, 1024, 640, D.DORA_BF16)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(y)
    W = torch.randn(640, 1024, device=DEV, dtype=BF)

    def step():
        D.dora_quantize_fourbit(W, codes=codes, scale=scale)
        D.dora_linear_fourbit(x, codes, scale, y=out, ws=ws)

    say("capture", T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        W.normal_()
        x.normal_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c, s = D.dora_quantize_fourbit(W)
        assert torch.equal(c, codes) and torch.equal(s, scale)
        assert torch.equal(out, D.dora_linear_fourbit(x, c, s))


def test_merged_weight_in_4_bits_between_the_norms():
    """As it is used: the merged weight in 4 bits behind the block norm, a decoded token at a
    time, against the same path on the restored weight."""
    g = torch.Generator().manual_seed(21)
    d, r = 512, 16
    W, A, B = (torch.randn(*s, generator=g).to(BF).to(DEV) * k
               for s, k in (((d, d), d ** -0.5), ((r, d), d ** -0.5), ((d, r), 0.02)))
    m = W.float().norm(dim=1) * 1.01
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).to(DEV)
    merged = D.dora_merge(W, A, B, m, 2.0)
    codes, scale = D.dora_quantize_fourbit(merged)
    restored = D.dora_dequantize_fourbit(codes, scale, d)
    for T in (1, 7, 100):
        x, res = (torch.randn(T, d, generator=g).to(BF).to(DEV) for _ in range(2))
        o = D.dora_block_norm(x, res, w, w_post=w)
        y = D.dora_linear_fourbit(o["y"], codes, scale)
        ref = o["y"].double().cpu() @ restored.double().cpu().T
        bound = (d + 8) * U * (o["y"].double().cpu().abs() @ restored.double().cpu().abs().T)
        assert ((y.cpu().double() - ref).abs() <= bound + ref.abs() * half(BF)).all()
        # e2m1 with a scale for 128 columns: a step is at most 1/3 of a value above 0.5 scale;
        # rows of normal weights come out about 0.12 off
        exact = o["y"].double().cpu() @ merged.double().cpu().T
        assert float((y.cpu().double() - exact).norm() / exact.norm()) < 0.25


def test_python_refuses():
    x = torch.zeros(4, 64, device=DEV, dtype=BF)
    codes, scale = D.dora_quantize_fourbit(x, group=32)
    for bad, call in (
            (ValueError, lambda: D.dora_quantize_fourbit(x, group=16)),
            (ValueError, lambda: D.dora_quantize_fourbit(x, group=0)),
            (ValueError, lambda: D.dora_quantize_fourbit(x[0])),
            (TypeError, lambda: D.dora_quantize_fourbit(x.half())),
            (ValueError, lambda: D.dora_quantize_fourbit(x.cpu())),
            (ValueError, lambda: D.dora_quantize_fourbit(x[:, ::2], group=32)),
            (ValueError, lambda: D.dora_dequantize_fourbit(codes, scale, 65, group=32)),
            (TypeError, lambda: D.dora_dequantize_fourbit(codes, scale.float(), 64, group=32)),
            (ValueError, lambda: D.dora_linear_fourbit(x, codes, scale, group=64)),
            (ValueError, lambda: D.dora_linear_fourbit(x[:, :32].contiguous(), codes, scale, group=32)),
            (TypeError, lambda: D.dora_linear_fourbit(x, codes.to(torch.int8), scale, group=32)),
            (TypeError, lambda: D.dora_linear_fourbit(x, codes, scale, group=32,
                                                      y=torch.empty(4, 4, device=DEV))),
            (D.DoraError, lambda: D.dora_linear_fourbit(
                torch.zeros(300, 64, device=DEV, dtype=BF), codes, scale, group=32,
                ws=torch.empty(16, dtype=torch.uint8, device=DEV)))):
        with pytest.raises(bad):
            call()
