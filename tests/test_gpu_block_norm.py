"""GPU: the norms on both sides of a residual addition and their gradients,
against their plain forms in 64 bits (the bounds, derived from the arithmetic,
stand with the plain forms in around_ref.py: sums of d terms (d / 64 + 64) u,
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
A, B = 0.875, 1.25


def draw(seed, T, d, dt, gate):
    """x, residual, w_post, gate, w_pre, dy, dh; gate: None, "channel", or tokens a gate row."""
    g = torch.Generator().manual_seed(seed)
    x, res, dy, dh = (torch.randn(T, d, generator=g) for _ in range(4))
    if d > 3:
        res[:, d // 3] *= 40.0
    w1, w2 = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    gt = None
    if gate is not None:
        gt = torch.randn(d if gate == "channel" else (T // gate, d), generator=g)
        gt = gt.reshape(d) if gate == "channel" else gt.reshape(T // gate, d)
    return [t if t is None else t.to(dt) for t in (x, res, w1, gt, w2, dy, dh)]


def up(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def within(got, ref, bound, what):
    got = got.cpu().double()
    assert got.shape == ref.shape, what
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert (off <= bound).all(), (f"{what}: {int((off > bound).sum())} of {off.numel()} off, worst "
                                  f"{float((off / bound.clamp_min(1e-300)).max()):.2f}x the bound")


def both(T, d, dt, gate, post=True, with_dh=True, seed=None, eps=1e-5, a=A, b=B):
    """Forward and backward, each against its plain form; returns what was computed."""
    seed = T * 100003 + d if seed is None else seed
    x, res, w1, gt, w2, dy, dh = draw(seed, T, d, dt, gate)
    w1 = w1 if post else None
    dh = dh if with_dh else None
    gx, gres, gw1, gg, gw2, gdy, gdh = up(x, res, w1, gt, w2, dy, dh)
    kw = {"w_post": gw1, "gate": gg, "residual_scale": a, "branch_scale": b}
    say("block norm", T, d, dt, gate, post, with_dh)
    o = D.dora_block_norm(gx, gres, gw2, eps=eps, want_rstd=True, **kw)
    h, bound = R.block_h(x, res, w1, gt, a, b, eps)
    within(o["h"], h, bound, "h")
    hs = o["h"].cpu()
    E = sum_error(d) + 3 * U
    r2 = R.rms_factor(hs, eps)
    within(o["rstd_pre"], r2, r2 * E, "rstd_pre")
    y = hs.double() * r2[:, None] * w2.double()
    within(o["y"], y, y.abs() * (E + 3 * U + half(dt)), "y")
    if post:
        r1 = R.rms_factor(x, eps)
        within(o["rstd_post"], r1, r1 * E, "rstd_post")
    say("block norm backward", T, d, dt, gate, post, with_dh)
    g = D.dora_block_norm_backward(gdy, gx, o["h"], gw2, o["rstd_pre"],
                                   rstd_post=o.get("rstd_post"), dh=gdh, **kw)
    ref = R.block_grad(dy, dh, x, hs, w2, o["rstd_pre"].cpu(), w1,
                       o["rstd_post"].cpu() if post else None, gt, a, b)
    assert set(g) == set(ref)
    for k, (v, e) in ref.items():
        within(g[k], v, e, k)
    return (gx, gres, gw1, gg, gw2, gdy, gdh), o, g


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 8), (6, 33), (4, 63), (8, 130), (16, 512), (36, 1027),
          (9, 2048), (6, 4099), (3, 8192), (2, 8200), (2, 16384), (2, 16387), (2, 28672),
          (1, 32775)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_matches_plain_form(T, d, dt):
    both(T, d, dt, "channel")
    both(T, d, dt, None, post=False, with_dh=False)
    both(T, d, dt, 1, with_dh=False)
    if T % 3 == 0:
        both(T, d, dt, 3)
        both(T, d, dt, 3, post=False)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d,gate", [
    (4096, 130, 2),        # gate rows inside a chunk: sums final there
    (4096, 130, 32),       # gate rows longer than a chunk: partial sums
    (3003, 65, 1001), (3003, 65, 7), (517, 2047, 47), (1030, 515, 5), (2056, 9, 257),
    (700, 8193, 35), (640, 16385, 2), (640, 16385, 64), (512, 1027, "channel"),
    (2000, 16390, "channel"), (1500, 24, "channel"), (300, 4100, 1)])
def test_many_rows(T, d, gate, dt):
    both(T, d, dt, gate)


@pytest.mark.parametrize("a,b", [(1.0, 1.0), (0.0, 2.0), (1.0, 0.0), (-0.5, -3.0)])
def test_scales(a, b):
    both(12, 300, BF, "channel", a=a, b=b)
    both(12, 300, F32, 4, a=a, b=b)


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("d", [520, 40000])
def test_in_place(d, T):
    if T == 600 and d == 40000:
        T = 60
    (x, res, w1, gt, w2, dy, dh), o, g = both(T, d, BF, "channel")
    kw = {"w_post": w1, "gate": gt, "residual_scale": A, "branch_scale": B}
    x2, r2 = x.clone(), res.clone()
    say("block norm in place", T, d)
    D.dora_block_norm(x2, r2, w2, eps=1e-5, out={"h": r2, "y": x2}, **kw)
    assert torch.equal(r2, o["h"]) and torch.equal(x2, o["y"])
    d2 = dh.clone()
    out = {"dx": torch.empty_like(x), "dresidual": d2}
    say("block norm backward in place", T, d)
    D.dora_block_norm_backward(dy, x, o["h"], w2, o["rstd_pre"], rstd_post=o["rstd_post"], dh=d2,
                               out=out, **kw)
    assert torch.equal(out["dx"], g["dx"]) and torch.equal(d2, g["dresidual"])


@pytest.mark.parametrize("dt", [BF, F32])
def test_no_tokens(dt):
    x = torch.empty(0, 70, dtype=dt, device=DEV)
    w = torch.ones(70, dtype=dt, device=DEV)
    r = torch.empty(0, device=DEV)
    for gate in (w, w.reshape(1, 70), None):
        say("no tokens", dt, None if gate is None else tuple(gate.shape))
        o = D.dora_block_norm(x, x, w, w_post=w, gate=gate, want_rstd=True)
        assert o["h"].shape == o["y"].shape == (0, 70)
        out = {"dx": x, "dresidual": x.clone(), "dw_pre": torch.full((70,), 7.0, device=DEV),
               "dw_post": torch.full((70,), 7.0, device=DEV)}
        if gate is not None:
            out["dgate"] = torch.full_like(gate, 7.0)
        D.dora_block_norm_backward(x, x, x, w, r, w_post=w, rstd_post=r, gate=gate, out=out)
        for k in ("dw_pre", "dw_post", "dgate"):
            if k in out:
                assert torch.count_nonzero(out[k]) == 0, k


@pytest.mark.parametrize("d", [300, 20000])
@pytest.mark.parametrize("dt", [BF, F32])
def test_zero_rows_and_nonfinite_rows(d, dt):
    x, res, w1, gt, w2, dy, dh = draw(5, 6, d, dt, "channel")
    x[1] = 0
    res[1] = 0
    x[2, 7] = float("inf")
    res[3, 9] = float("nan")
    gx, gres, gw1, gg, gw2 = up(x, res, w1, gt, w2)
    say("zero and non-finite rows", d, dt)
    o = D.dora_block_norm(gx, gres, gw2, w_post=gw1, gate=gg, eps=1e-5)
    assert torch.count_nonzero(o["h"][1]) == 0 and torch.count_nonzero(o["y"][1]) == 0
    assert o["y"][2].isnan().any() and o["y"][3].isnan().all()
    fine = [0, 4, 5]
    h, bound = R.block_h(x[fine], res[fine], w1, gt, 1.0, 1.0, 1e-5)
    within(o["h"][fine], h, bound, "h beside them")
    assert o["y"][fine].isfinite().all()


@pytest.mark.parametrize("d", [129, 17000])
@pytest.mark.parametrize("power", [-70, -40, 40, 70])
def test_rows_of_any_magnitude(power, d):
    """hat(x) and hat(h) do not depend on the rows' magnitude, nor do relative errors."""
    k = 2.0 ** power
    x, res, w1, gt, w2, dy, _ = draw(9, 5, d, F32, "channel")
    x, res = x * k, res * k
    gx, gres, gw1, gg, gw2, gdy = up(x, res, w1, gt, w2, dy)
    say("rows of 2^", power, d)
    kw = {"w_post": gw1, "gate": gg, "residual_scale": A, "branch_scale": B * k}
    o = D.dora_block_norm(gx, gres, gw2, eps=0.0, want_rstd=True, **kw)
    h, bound = R.block_h(x, res, w1, gt, A, B * k, 0.0)
    within(o["h"], h, bound, "h")
    hs = o["h"].cpu()
    r2 = R.rms_factor(hs, 0.0)
    y = hs.double() * r2[:, None] * w2.double()
    within(o["y"], y, y.abs() * (sum_error(d) + 6 * U + half(F32)), "y")
    g = D.dora_block_norm_backward(gdy, gx, o["h"], gw2, o["rstd_pre"], rstd_post=o["rstd_post"], **kw)
    ref = R.block_grad(dy, None, x, hs, w2, o["rstd_pre"].cpu(), w1, o["rstd_post"].cpu(), gt, A, B * k)
    for name, (v, e) in ref.items():
        within(g[name], v, e, name)


def test_streams_and_repeats_give_the_same_bits():
    (x, res, w1, gt, w2, dy, dh), o, g = both(400, 3000, BF, "channel")
    kw = {"w_post": w1, "gate": gt, "residual_scale": A, "branch_scale": B}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(D.dora_block_norm_backward(dy, x, o["h"], w2, o["rstd_pre"], dh=dh,
                                                   rstd_post=o["rstd_post"], **kw))
    torch.cuda.synchronize()
    for other in outs:
        for k in g:
            assert torch.equal(other[k], g[k]), k


@pytest.mark.parametrize("gate", ["channel", 1, 50])
def test_captured_and_replayed(gate):
    (x, res, w1, gt, w2, dy, dh), o, g = both(200, 1000, BF, gate)
    kw = {"w_post": w1, "gate": gt, "residual_scale": A, "branch_scale": B}
    fo = {k: torch.empty_like(v) for k, v in o.items()}
    go = {k: torch.empty_like(v) for k, v in g.items()}
    ws = torch.empty(D.dora_block_norm_backward_workspace(
        200, 1000, {"channel": 200, 1: 1, 50: 50}[gate], D.DORA_BF16) + 16, dtype=torch.uint8,
        device=DEV)

    def step():
        D.dora_block_norm(x, res, w2, eps=1e-5, out=fo, **kw)
        D.dora_block_norm_backward(dy, x, fo["h"], w2, fo["rstd_pre"], rstd_post=fo["rstd_post"],
                                   dh=dh, ws=ws, out=go, **kw)

    say("capture", gate)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x2, res2, _, _, _, dy2, dh2 = up(*draw(70 + k, 200, 1000, BF, None))
        x.copy_(x2), res.copy_(res2), dy.copy_(dy2), dh.copy_(dh2)
        for t in (*fo.values(), *go.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        e = D.dora_block_norm(x, res, w2, eps=1e-5, want_rstd=True, **kw)
        eg = D.dora_block_norm_backward(dy, x, e["h"], w2, e["rstd_pre"], rstd_post=e["rstd_post"],
                                        dh=dh, **kw)
        for name in e:
            assert torch.equal(fo[name], e[name]), name
        for name in eg:
            assert torch.equal(go[name], eg[name]), name


def test_offsets_past_32_bits():
    """The rows behind the first 2^31 elements."""
    T, d = (1 << 31) // 4096 + 5, 4096
    say("block norm past 2^31 elements")
    g = torch.Generator(DEV).manual_seed(2)
    x = torch.randn(T, d, device=DEV, dtype=BF, generator=g)
    w = torch.ones(d, device=DEV, dtype=BF)
    res = x.flip(1)
    o = D.dora_block_norm(x, res, w, w_post=w, gate=x, want_rstd=True)
    tail = slice(T - 4, T)
    xs, rs, ws = x[tail].cpu(), res[tail].cpu(), w.cpu()
    h, bound = R.block_h(xs, rs, ws, xs, 1.0, 1.0, 1e-6)
    within(o["h"][tail], h, bound, "h")
    hs = o["h"][tail].cpu()
    r2 = R.rms_factor(hs, 1e-6)
    y = hs.double() * r2[:, None]
    within(o["y"][tail], y, y.abs() * (sum_error(d) + 6 * U + half(BF)), "y")
    gr = D.dora_block_norm_backward(res, x, o["h"], w, o["rstd_pre"], w_post=w,
                                    rstd_post=o["rstd_post"], gate=x, dh=x)
    ref = R.block_grad(rs, xs, xs, hs, ws, o["rstd_pre"][tail].cpu(), ws,
                       o["rstd_post"][tail].cpu(), xs, 1.0, 1.0)
    for k in ("dx", "dresidual", "dgate"):
        within(gr[k][tail], *ref[k], k)


def test_python_refuses():
    x = torch.zeros(6, 64, device=DEV, dtype=BF)
    w = torch.ones(64, device=DEV, dtype=BF)
    r = torch.ones(6, device=DEV)
    for bad, kw in ((ValueError, {"gate": torch.ones(4, 64, device=DEV, dtype=BF)}),
                    (ValueError, {"gate": torch.ones(6, 63, device=DEV, dtype=BF)}),
                    (ValueError, {"gate": torch.ones(12, 64, device=DEV, dtype=BF)}),
                    (TypeError, {"gate": torch.ones(64, device=DEV)}),
                    (TypeError, {"w_post": torch.ones(64, device=DEV)}),
                    (ValueError, {"w_post": torch.ones(32, device=DEV, dtype=BF)}),
                    (ValueError, {"out": {"h": x.clone()}}),
                    (ValueError, {"out": {"h": x.clone(), "y": x.clone(), "q": x}}),
                    (D.DoraError, {"out": {"h": x, "y": x}}),
                    (D.DoraError, {"eps": -1.0}), (D.DoraError, {"branch_scale": float("nan")})):
        with pytest.raises(bad):
            D.dora_block_norm(x, x.clone(), w, **kw)
    with pytest.raises(ValueError):
        D.dora_block_norm(x, x[:3].clone(), w)
    with pytest.raises(ValueError):
        D.dora_block_norm(x.cpu(), x, w)
    with pytest.raises(ValueError):
        D.dora_block_norm(x[:, ::2], x[:, ::2], w[::2])
    with pytest.raises(ValueError):
        D.dora_block_norm_backward(x, x, x, w, r, w_post=w)
    with pytest.raises(ValueError):
        D.dora_block_norm_backward(x, x, x, w, r, out={"dx": x.clone()})
    with pytest.raises(ValueError):
        D.dora_block_norm_backward(x, x, x, w, r, out={"dx": x.clone(), "dresidual": x.clone(),
                                                       "dgate": x.clone()})
    with pytest.raises(D.DoraError):
        D.dora_block_norm_backward(x, x.clone(), x.clone(), w, r, out={"dx": x, "dresidual": x.clone()})
    with pytest.raises(D.DoraError):
        D.dora_block_norm_backward(torch.zeros(600, 64, device=DEV, dtype=BF),
                                   torch.zeros(600, 64, device=DEV, dtype=BF),
                                   torch.zeros(600, 64, device=DEV, dtype=BF), w,
                                   torch.ones(600, device=DEV),
                                   ws=torch.empty(16, dtype=torch.uint8, device=DEV))
