"""GPU: block norms of rows whose squares leave fp32's range, next to ordinary
ones, over several waves: the sums of x's squares, of h's, and their second
passes over scaled values keep to LDS rows of their own.

Bounds as in test_gpu_block_norm.py (sums of d terms (d / 64 + 64) u,
u = 2^-24, a few u for each product, half a step of the output's type)."""
import pytest
import torch

import around_ref as R
from around_ref import U, half, sum_error
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# what a row of x, and one of the residual, is scaled by: with eps = 0 powers of 70 and -70 take
# the second pass, of x's sum alone, of h's alone, and of both
POWERS = [(0, 0), (70, 0), (-70, 0), (0, 70), (70, 70), (-70, -70), (0, -70), (-70, 70), (70, -70)]


def rows(seed, T, d, dt):
    g = torch.Generator().manual_seed(seed)
    x, res = torch.randn(T, d, generator=g), torch.randn(T, d, generator=g)
    w1, w2 = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    # the branch as large as the residual stream, so that h takes the magnitude of either
    gate = torch.ones(T, d)
    for t in range(T):
        a, b = POWERS[t % len(POWERS)]
        x[t] *= 2.0 ** a
        res[t] *= 2.0 ** b
        gate[t] *= 2.0 ** b
    return [v.to(dt) for v in (x, res, w1, w2, gate)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", [(9, 129), (18, 1024), (36, 4096), (27, 8192), (540, 8192), (540, 5003),
                                 (18, 16384), (18, 32768)])
def test_ordinary_and_rescaled_rows_side_by_side(T, d, dt):
    x, res, w1, w2, gate = rows(T + d, T, d, dt)
    gx, gres, gw1, gw2, gg = (v.to(DEV) for v in (x, res, w1, w2, gate))
    say("ordinary and rescaled rows", T, d, dt)
    o = D.dora_block_norm(gx, gres, gw2, w_post=gw1, gate=gg, eps=0.0, want_rstd=True)
    h, bound = R.block_h(x, res, w1, gate, 1.0, 1.0, 0.0)
    hs = o["h"].cpu()
    assert ((hs.double() - h).abs() <= bound).all()
    E = sum_error(d) + 3 * U
    for name, of in (("rstd_post", x), ("rstd_pre", hs)):
        r = R.rms_factor(of, 0.0)
        assert ((o[name].cpu().double() - r).abs() <= r * E).all(), name
    y = hs.double() * R.rms_factor(hs, 0.0)[:, None] * w2.double()
    assert ((o["y"].cpu().double() - y).abs() <= y.abs() * (E + 3 * U + half(dt))).all()
    # each row as it is by itself
    for t in (0, 1, 4, 5):
        one = D.dora_block_norm(gx[t:t + 1].clone(), gres[t:t + 1].clone(), gw2, w_post=gw1,
                                gate=gg[t:t + 1].clone(), eps=0.0, want_rstd=True)
        if T <= 512:  # (the same number of vectors a thread, so the same sums)
            for name in o:
                assert torch.equal(one[name], o[name][t:t + 1]), (name, t)
