"""GPU: dA of the backward from 8-bit checkpoints, from x's int8 rows themselves (bf16,
one scale a row or groups of 128 columns and more).

With g = m / n = 1 and yq = 0 (dm = 0, so the norm's part of the gradient is 0) dh = dy
and nothing of dA = Q^T x, Q = s dy B, is rounded to bf16 but dA itself.  Bounds
(u = 2^-8 half a step of bf16, relative): u |dA|; the pair of bf16 that Q xs becomes
keeps it to u^2 = 2^-16; every fp32 sum adds 2^-23 a term of its absolute terms, of
d_out terms (Q) and T (dA).  A Q or x rounded to bf16 would be off by
up to u |Q|^T |x|, which the sum over tokens does not cancel as dA does."""
import pytest
import torch

import rows8_ref as R
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
U = 2.0 ** -8


def operands(T, d_in, d_out, r, group, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dy, W, A, B = rnd(T, d_out), rnd(d_out, d_in) / 8, rnd(r, d_in) / 8, rnd(d_out, r) / 4
    x = rnd(T, d_in) * torch.exp(rnd(T, 1))
    xq, xs = R.quantize(x, group)
    n = 1 if group == 0 else -(-d_out // group)
    yq, ys = torch.zeros(T, d_out, dtype=torch.int8), torch.ones(T, n)
    return [t.to(BF) for t in (dy, W, A, B)] + [xq, xs, yq, ys]


def call(ops, s, group, through, **kw):
    dy, W, A, B, xq, xs, yq, ys = [t.to(DEV) for t in ops]
    one = torch.ones(W.shape[0], device=DEV)
    P = torch.zeros(dy.shape[0], A.shape[0], dtype=BF, device=DEV)
    return D.dora_backward_checkpoint(dy, xq, xs, W, A, B, one, one, s, P, yq, ys, group=group,
                                      through_norm=through, **kw)


def check(ops, s, group, through, got):
    dy, W, A, B, xq, xs, _, _ = ops
    T, d_out = dy.shape
    d_in = xq.shape[1]
    x = xq.double() * R.spread(xs, d_in, group)
    Q = s * dy.double() @ B.double()
    ref = Q.T @ x
    f32 = (T + 4) * 2.0 ** -23
    sums = abs(s) * dy.double().abs() @ B.double().abs()
    bound = (U * ref.abs() + ((U * U + f32) * Q.abs() + (d_out + 4) * 2.0 ** -23 * sums).T @ x.abs())
    off = (got["dA"].cpu().double() - ref).abs()
    assert (off <= bound * (1 + 1e-6) + 1e-38).all(), (
        f"{int((off > bound).sum())} of {off.numel()} off, worst {float((off / bound).max()):.2f}x")
    assert (got["dm"] == 0).all()


# tokens, widths and ranks at and beside the tile (64 x 128), the step (64 tokens) and the
# eight columns of a chunk; splits of K
SIZES = [(1, 1, 8, 1), (2, 7, 3, 2), (5, 8, 16, 9), (63, 130, 40, 64), (64, 128, 64, 65),
         (65, 127, 33, 63), (129, 256, 128, 128), (300, 1027, 72, 37), (1000, 136, 264, 5),
         (2049, 515, 96, 130), (4096, 384, 48, 200)]


@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("T,d_in,d_out,r", SIZES)
def test_dA_of_8_bit_rows_is_rounded_once(T, d_in, d_out, r, through):
    for group in (0, 128, 256, 512):
        ops = operands(T, d_in, d_out, r, group, T + d_in + group)
        say("dA from 8 bits", T, d_in, d_out, r, group, through)
        check(ops, 1.5, group, through, call(ops, 1.5, group, through))


def test_dA_norm_is_that_of_its_own_rounding_and_dhs():
    """With g other than 1: half a step's rms, 2^-8 / sqrt 3 of random mantissas at
    most 0.0017, for each of dA's and dh's roundings, and nothing else."""
    T, d_in, d_out, r = 512, 640, 512, 48
    for group in (0, 128):
        ops = operands(T, d_in, d_out, r, group, 3)
        dy, W, A, B, xq, xs, yq, ys = ops
        m = torch.rand(d_out, generator=torch.Generator().manual_seed(4)) + 0.5
        dev = [t.to(DEV) for t in ops]
        say("dA's norm error", group)
        got = D.dora_backward_checkpoint(dev[0], dev[4], dev[5], *dev[1:4], m.to(DEV),
                                         torch.ones(d_out, device=DEV), 1.0,
                                         torch.zeros(T, r, dtype=BF, device=DEV), dev[6], dev[7],
                                         group=group)
        Q = (dy.double() * m.double()) @ B.double()
        ref = Q.T @ (xq.double() * R.spread(xs, d_in, group))
        rel = float((got["dA"].cpu().double() - ref).norm() / ref.norm())
        assert rel <= 0.0017 * 2 ** 0.5 * 1.03, rel


@pytest.mark.parametrize("through", [False, True])
def test_scales_of_any_size_zeros_and_nan(through):
    ops = operands(200, 260, 48, 20, 128, 5)
    ops[5] = ops[5] * 2.0 ** torch.linspace(-60, 60, 200)[:, None]
    say("dA from 8 bits, scales far apart")
    check(ops, 1.0, 128, through, call(ops, 1.0, 128, through))
    ops[5][7] = 0
    ops[5][9, 1] = float("nan")
    say("dA from 8 bits, a zero and a NaN scale")
    got = call(ops, 1.0, 128, through)["dA"].cpu()
    # the NaN's group of columns only
    assert torch.isnan(got[:, 128:256]).all()
    assert torch.isfinite(got[:, :128]).all() and torch.isfinite(got[:, 256:]).all()


@pytest.mark.parametrize("ex,eq", [(-118, 100), (-126, 60), (110, -110), (90, -100), (-60, -40), (-120, 118)])
def test_rows_and_gradients_far_from_one(ex, eq):
    """Scales and Q of which one is far below and the other far above one, or whose
    product is near the smallest normal number: dA is right to its own rounding."""
    ops = operands(300, 260, 48, 20, 128, 8)
    ops[5] = (ops[5] / ops[5].max() * 2.0 ** ex).clamp_min(2.0 ** -126)
    ops[0] = (ops[0].float() * 2.0 ** eq).to(BF)
    say("dA from 8 bits, scales of 2^%d, dy of 2^%d" % (ex, eq))
    check(ops, 1.0, 128, False, call(ops, 1.0, 128, False))


def test_an_infinite_gradient_stays_one():
    ops = operands(70, 136, 16, 8, 0, 6)
    ops[0][3] = 3.0e38  # Q of token 3 overflows
    ops[3][:] = ops[3].abs() + 1
    ops[4][3] = 5
    say("dA from 8 bits, an infinite Q")
    assert (call(ops, 1.0, 0, False)["dA"] == float("inf")).all()


def test_one_workspace_for_every_group():
    """One workspace serves calls of every group, one after the other."""
    T, d_in, d_out, r = 150, 270, 64, 24
    ws = torch.empty(D.dora_backward_checkpoint_workspace(T, d_in, d_out, r, D.DORA_BF16),
                     dtype=torch.uint8, device=DEV)
    for group in (128, 32, 0, 64, 512):
        ops = operands(T, d_in, d_out, r, group, 7 + group)
        say("one workspace", group)
        a, b = call(ops, 1.0, group, False, ws=ws), call(ops, 1.0, group, False)
        for k in a:
            assert torch.equal(a[k], b[k]), (group, k)
        if group % 128 == 0:
            check(ops, 1.0, group, False, a)


@pytest.mark.parametrize("through", [False, True])
def test_captured_replayed_and_on_a_second_stream(through):
    """Replays on other inputs, with eager work between them, give the eager bits; so
    does a call on a stream of its own beside one on another."""
    T, d_in, d_out, r, group = 190, 270, 200, 40, 128
    dev = [t.to(DEV) for t in operands(T, d_in, d_out, r, group, 11)]
    dy, W, A, B, xq, xs, yq, ys = dev
    gen = torch.Generator(DEV).manual_seed(12)
    m = torch.rand(d_out, generator=gen, device=DEV) + 0.5
    n = torch.rand(d_out, generator=gen, device=DEV) + 0.5
    P = torch.randn(T, r, generator=gen, device=DEV).to(BF)
    yq.copy_(torch.randint(-127, 128, (T, d_out), generator=gen, device=DEV, dtype=torch.int8))

    def step():
        return D.dora_backward_checkpoint(dy, xq, xs, W, A, B, m, n, 1.25, P, yq, ys, group=group,
                                          through_norm=through)

    say("dA from 8 bits, two streams", through)
    eager = step()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st in (a, b):
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(o[k], eager[k]) for k in eager)
    say("dA from 8 bits, capture", through)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in range(4):
        if k:
            dy.copy_(torch.randn(T, d_out, generator=gen, device=DEV))
            xq.copy_(torch.randint(-127, 128, (T, d_in), generator=gen, device=DEV, dtype=torch.int8))
            xs.copy_(torch.rand(xs.shape, generator=gen, device=DEV))
        say("replay", k)
        graph.replay()
        torch.cuda.synchronize()
        copy = {key: v.clone() for key, v in kept.items()}
        now = step()
        torch.cuda.synchronize()
        for key in now:
            assert torch.equal(copy[key], now[key]), (k, key)


def test_offsets_past_32_bits():
    """2.2e9 int8 values of x; whole numbers, so that every sum is exact."""
    T, d_in, d_out, r = 66_001, 32_776, 8, 3
    g = torch.Generator(DEV).manual_seed(1)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV).to(BF)  # noqa: E731
    dy, W, A, B, P = ints(T, d_out), ints(d_out, d_in), ints(r, d_in), ints(d_out, r), ints(T, r)
    xq = torch.randint(-127, 128, (T, d_in), generator=g, device=DEV, dtype=torch.int8)
    for group in (0, 128):
        one = torch.ones(d_out, device=DEV)
        xs = torch.ones(T, 1 if group == 0 else -(-d_in // group), device=DEV)
        yq, ys = torch.zeros(T, d_out, dtype=torch.int8, device=DEV), torch.ones(T, 1, device=DEV)
        say("dA from 8 bits, past 32 bits", group)
        got = D.dora_backward_checkpoint(dy, xq, xs, W, A, B, one, one, 1.0, P, yq, ys, group=group)
        Q = dy.cpu().double() @ B.cpu().double()
        at = torch.tensor([0, 1, 127, 128, 16_000, d_in - 9, d_in - 8, d_in - 1])
        want = Q.T @ xq[:, at.to(DEV)].cpu().double()
        assert want.abs().max() < 2 ** 23
        assert torch.equal(got["dA"][:, at.to(DEV)].cpu(), want.to(BF)), group
        rows = torch.tensor([0, 40_000, 65_535, 65_536, T - 1])
        full = dy[rows.to(DEV)].cpu().double() @ W.cpu().double() + Q[rows] @ A.cpu().double()
        assert torch.equal(got["dx"][rows.to(DEV)].cpu(), full.to(BF))
        del got
