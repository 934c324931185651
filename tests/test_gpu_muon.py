"""GPU: matrices orthogonalised by Newton-Schulz steps and the optimiser's step,
against the literal steps in 64 bits.  Bounds in the Frobenius norm, derived
with the plain form (orthogonal_bound in around_ref.py); the momentum is two
fp32 roundings off, element by element."""
import pytest
import torch

import around_ref as R
from around_ref import U as EPS32
from around_ref import half
from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def matrix(seed, rows, cols, dt, fall=0.5, size=1.0):
    """Singular values that fall off over a floor of noise."""
    g = torch.Generator().manual_seed(seed)
    k = min(rows, cols)
    left, right = torch.randn(rows, k, generator=g), torch.randn(k, cols, generator=g)
    U = (left * torch.arange(1, k + 1).float() ** -fall) @ right
    return ((U + 0.05 * torch.randn(rows, cols, generator=g)) * size).to(dt)


def check(U, **kw):
    say("orthogonalize", tuple(U.shape), U.dtype, kw)
    O = D.dora_orthogonalize(U.to(DEV), **kw).cpu()
    assert O.dtype == U.dtype
    ref = R.orthogonal(U, **kw)
    off = float(torch.linalg.vector_norm(O.double() - ref))
    bound = R.orthogonal_bound(U, ref, U.dtype, **kw)
    assert off <= bound, f"off by {off:.3e}, bound {bound:.3e}"
    return O, ref


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (8, 8), (37, 1027), (1027, 37), (16, 4096), (64, 2000),
          (2000, 64), (65, 300), (300, 65), (128, 1024), (129, 130), (200, 200), (1500, 384),
          (384, 1500), (257, 255)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dt):
    for fall in (0.0, 1.0):
        check(matrix(rows * 7 + cols, rows, cols, dt, fall))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 9])
def test_steps_and_coefficients(steps, dt):
    for n in (20, 100):
        check(matrix(n, n, 333, dt), steps=steps)
        # the cubic steps, and others
        check(matrix(n, 333, n, dt), steps=steps, coefficients=(1.5, -0.5, 0.0))
        check(matrix(n, n, 333, dt), steps=steps, coefficients=(2.0, -1.5, 0.5), eps=0.1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("power", [-110, -60, -20, 60, 100])
def test_any_magnitude(power, dt):
    """O does not depend on U's magnitude (eps = 0), though its squares leave fp32's range."""
    for shape in ((30, 700), (700, 150)):
        U = matrix(5, *shape, dt)
        check((U.double() * 2.0 ** power).to(dt), eps=0.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", [(30, 700), (700, 150)])
def test_norms_at_the_ends_of_the_range(shape, dt):
    """|U| of 2^-117 and 2^126 or so: 1 / |U| times Q's elements would leave fp32's range."""
    for power in (-126, -122, -118, 110, 114, 118):
        U = matrix(5, *shape, F32).to(dt).double() * 2.0 ** power
        assert float(U.abs().max()) < 2.0 ** 127
        check(U.to(dt), eps=0.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_zeros_stay_zeros_whatever_eps(dt):
    for shape in ((30, 700), (700, 150)):
        for eps in (1e-7, 1e-37, 2e-38):
            O = D.dora_orthogonalize(torch.zeros(*shape, dtype=dt, device=DEV), eps=eps)
            assert torch.count_nonzero(O) == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("powers", [(-100, 0, 90), (90, 0, -100), (None, -100, -100), (None, None, 0),
                                    (0, -100, None), (-100, -90, -80)])
def test_magnitudes_that_change_along_the_longer_side(powers, dt):
    """Whole stretches far below the others, or of zeros."""
    for n, length in ((30, 9000), (61, 2050), (150, 2100)):
        U = matrix(n, n, length, dt).double()
        for k, power in enumerate(powers):
            U[:, length * k // 3:length * (k + 1) // 3] *= 0.0 if power is None else 2.0 ** power
        check(U.to(dt), eps=0.0)
        check(U.T.contiguous().to(dt), eps=0.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,length", [(20, 40001), (64, 33000), (33, 40000)])
def test_long_and_narrow(n, length, dt):
    check(matrix(n, n, length, dt, fall=0.2))
    check(matrix(n, length, n, dt, fall=0.2))


def test_singular_values_come_close_to_one():
    """Each one becomes what the steps make of it (two matrices' singular values differ by no
    more than the matrices do)."""
    U = matrix(3, 96, 2048, F32, fall=0.2)
    O, ref = check(U)
    f = torch.linalg.svdvals(U.double()) / torch.linalg.vector_norm(U.double())
    big = f >= 2e-3
    a, b, c = R.QUINTIC
    for _ in range(5):
        f = a * f + b * f ** 3 + c * f ** 5
    s = torch.linalg.svdvals(O.double())
    assert float((s - f.sort(descending=True)[0]).abs().max()) <= R.orthogonal_bound(U, ref, F32) + 1e-9
    assert 0.67 < float(f[big].min()) and float(f[big].max()) < 1.21


@pytest.mark.parametrize("dt", [BF, F32])
def test_zeros_nonfinite_and_in_place(dt):
    for shape in ((20, 300), (400, 130)):
        z = torch.zeros(*shape, dtype=dt, device=DEV)
        assert torch.count_nonzero(D.dora_orthogonalize(z)) == 0
        U = matrix(8, *shape, dt).to(DEV)
        want = D.dora_orthogonalize(U)
        V = U.clone()
        assert D.dora_orthogonalize(V, out=V) is V and torch.equal(V, want)
        for bad in (float("nan"), float("inf")):
            V = U.clone()
            V[3, 5] = bad
            assert D.dora_orthogonalize(V).isnan().all()


def problem(shapes, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    ps = [(torch.randn(*s, generator=g) * s[1] ** -0.5).to(dt) for s in shapes]
    gs = [matrix(seed + 10 * k, *s, dt, size=1e-3) for k, s in enumerate(shapes)]
    ms = [matrix(seed + 10 * k + 5, *s, F32, size=3e-3) for k, s in enumerate(shapes)]
    return ps, gs, ms


def check_step(ps, gs, ms, out, new, lr, mu=0.95, decay=0.0, scales=None, nesterov=True, **kw):
    for k, (p, g, m) in enumerate(zip(ps, gs, ms)):
        dt, scale = p.dtype, 1.0 if scales is None else scales[k]
        mu32, lr32 = float(torch.tensor(mu)), float(torch.tensor(lr))
        m1 = mu32 * m.double() + g.double()
        off = (new[k].cpu().double() - m1).abs()
        assert (off <= 2 * EPS32 * ((mu32 * m.double()).abs() + m1.abs())).all(), k
        U = g.double() + mu32 * m1 if nesterov else m1
        O = R.orthogonal(U, **kw)
        ref = p.double() - lr32 * (decay * p.double() + scale * O)
        # U itself is a few fp32 roundings of its terms off
        terms = g.double().abs() + 2 * (mu32 * m1).abs() + 2 * (mu32 * m.double()).abs()
        moved = 3 * EPS32 * float(torch.linalg.vector_norm(terms) / torch.linalg.vector_norm(U))
        bound = abs(lr32 * scale) * R.orthogonal_bound(U, O, dt, moved=moved, **kw) \
            + float(torch.linalg.vector_norm(ref.abs() * half(dt))) \
            + 8 * EPS32 * float(torch.linalg.vector_norm(p.double().abs() + lr32 * scale * O.abs()))
        d = float(torch.linalg.vector_norm(out[k].cpu().double() - ref))
        assert d <= bound, f"matrix {k} {tuple(p.shape)}: off by {d:.3e}, bound {bound:.3e}"


LISTS = [[(16, 256)], [(384, 512), (700, 384)], [(37, 515), (1027, 37), (1, 9), (130, 64), (64, 64)],
         [(8, 300), (300, 8)] * 10, [(100, 40), (40, 100), (200, 150), (150, 200)] * 5]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("which", range(len(LISTS)))
def test_muon(which, dt):
    ps, gs, ms = problem(LISTS[which], dt, seed=which)
    up = [[t.to(DEV) for t in ts] for ts in (ps, gs, ms)]
    n = len(ps)
    scales = [0.2 * max(p.shape) ** 0.5 for p in ps]
    for kw in ({"mu": 0.95, "decay": 0.1, "nesterov": True}, {"mu": 0.8, "decay": 0.0, "nesterov": False}):
        say("muon", LISTS[which][:4], dt, kw)
        po, mo = [torch.empty_like(t) for t in up[0]], [torch.empty_like(t) for t in up[2]]
        D.dora_muon(*up, 0.02, mu=kw["mu"], weight_decay=kw["decay"], scales=scales,
                    nesterov=kw["nesterov"], params_out=po, momenta_out=mo)
        check_step(ps, gs, ms, po, mo, 0.02, scales=scales, **kw)
    # in place: the same bits
    p2, m2 = [t.clone() for t in up[0]], [t.clone() for t in up[2]]
    back = D.dora_muon(p2, up[1], m2, 0.02, mu=0.8, scales=scales, nesterov=False)
    assert back[0] is p2 and back[1] is m2
    for k in range(n):
        assert torch.equal(p2[k], po[k]) and torch.equal(m2[k], mo[k]), k


@pytest.mark.parametrize("shapes", [[(8, 300), (300, 8), (70, 90)] * 30, [(33, 200000), (200000, 9)] * 4])
@pytest.mark.parametrize("dt", [BF, F32])
def test_more_than_one_set_of_launches(shapes, dt):
    """More matrices than share a launch, and more bytes."""
    ps, gs, ms = problem(shapes, dt, seed=3)
    up = [[t.to(DEV) for t in ts] for ts in (ps, gs, ms)]
    po, mo = p2(up[0]), p2(up[2])
    D.dora_muon(*up, 0.02, params_out=po, momenta_out=mo)
    check_step(ps, gs, ms, po, mo, 0.02)
    again, m2 = p2(up[0]), p2(up[2])
    D.dora_muon(*up, 0.02, params_out=again, momenta_out=m2)
    assert all(torch.equal(x, y) for x, y in zip(again + m2, po + mo))


def test_a_matrix_does_not_depend_on_its_neighbours():
    """(Beyond the order of its sums, which its share of the launch decides.)"""
    ps, gs, ms = problem([(48, 900), (260, 70), (48, 900)], F32, seed=4)
    for t in (ps, gs, ms):
        t[2] = t[0].clone()
    up = [[t.to(DEV) for t in ts] for ts in (ps, gs, ms)]
    po, mo = [torch.empty_like(t) for t in up[0]], [torch.empty_like(t) for t in up[2]]
    D.dora_muon(*up, 0.02, params_out=po, momenta_out=mo)
    assert torch.equal(po[0], po[2]) and torch.equal(mo[0], mo[2])
    gs[1][3, 3] = float("nan")
    D.dora_muon(up[0], [g.to(DEV) for g in gs], up[2], 0.02, params_out=p2(po), momenta_out=p2(mo))
    check_step(ps[:1], gs[:1], ms[:1], po, mo, 0.02)


def p2(ts):
    return [torch.empty_like(t) for t in ts]


def test_training_step_of_a_module_between_norms():
    """As it is used: the block norm, the module, their gradients, and the factors' step."""
    g = torch.Generator().manual_seed(31)
    T, d, r = 192, 256, 16
    W, A, Bf = (torch.randn(*s, generator=g).to(DEV) * k
                for s, k in (((d, d), d ** -0.5), ((r, d), d ** -0.5), ((d, r), 0.02)))
    m = W.norm(dim=1) * 1.01
    w = 1 + 0.1 * torch.randn(d, generator=g).to(DEV)
    x, res, dy = (torch.randn(T, d, generator=g).to(DEV) for _ in range(3))
    o = D.dora_block_norm(x, res, w, w_post=w, want_rstd=True)
    y, n, P = D.dora_forward(o["y"], W, A, Bf, m, 2.0)
    b = D.dora_backward(dy, o["y"], W, A, Bf, m, n, 2.0, P, y)
    back = D.dora_block_norm_backward(b["dx"], x, o["h"], w, o["rstd_pre"], w_post=w,
                                      rstd_post=o["rstd_post"], dh=dy)
    momenta = [torch.zeros_like(A), torch.zeros_like(Bf)]
    before = [A.cpu().clone(), Bf.cpu().clone()]
    D.dora_muon([A, Bf], [b["dA"], b["dB"]], momenta, 0.02, scales=[0.5, 0.5])
    check_step(before, [b["dA"].cpu(), b["dB"].cpu()], [torch.zeros(r, d), torch.zeros(d, r)],
               [A, Bf], momenta, 0.02, scales=[0.5, 0.5])
    # the same step by differentiation in 64 bits, the norm n held
    leaf = [t.double().cpu().requires_grad_() for t in (x, res, before[0], before[1])]
    X, Rs, A64, B64 = leaf
    w64 = w.double().cpu()
    h = Rs + X * ((X * X).mean(1, keepdim=True) + 1e-6).rsqrt() * w64
    v = h * ((h * h).mean(1, keepdim=True) + 1e-6).rsqrt() * w64
    g64 = (m.double() / n.double()).cpu()
    out = g64 * (v @ W.double().cpu().T + 2.0 * (v @ A64.T) @ B64.T)
    ((out + h) * dy.double().cpu()).sum().backward()
    for name, got, t in (("dx", back["dx"], X), ("dresidual", back["dresidual"], Rs),
                         ("dA", b["dA"], A64), ("dB", b["dB"], B64)):
        ref = t.grad
        rel = float((got.double().cpu() - ref).norm() / ref.norm())
        assert rel < 1e-5, (name, rel)  # (fp32 modules: 1e-5 of the norm, as for each gradient)


@pytest.mark.parametrize("dt", [BF, F32])
def test_streams_and_graphs(dt):
    shapes = [(24, 500), (500, 24), (140, 300)]
    ps, gs, ms = problem(shapes, dt, seed=9)
    up = [[t.to(DEV) for t in ts] for ts in (ps, gs, ms)]
    want = D.dora_muon(*up, 0.02, params_out=p2(up[0]), momenta_out=p2(up[2]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(D.dora_muon(*up, 0.02, params_out=p2(up[0]), momenta_out=p2(up[2])))
    torch.cuda.synchronize()
    for o in outs:
        for k in range(3):
            assert torch.equal(o[0][k], want[0][k]) and torch.equal(o[1][k], want[1][k])
    ws = torch.empty(D.dora_muon_workspace(up[0]), dtype=torch.uint8, device=DEV)
    O = torch.empty_like(up[1][2])
    ws2 = torch.empty(D.dora_orthogonalize_workspace(140, 300, D.DORA_BF16 if dt == BF else D.DORA_F32),
                      dtype=torch.uint8, device=DEV)
    po, mo = p2(up[0]), p2(up[2])

    def step():
        D.dora_muon(*up, 0.02, params_out=po, momenta_out=mo, ws=ws)
        D.dora_orthogonalize(up[1][2], out=O, ws=ws2)

    say("capture", dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in up[1]:
            t.normal_()
        ws.fill_(0xFF), ws2.fill_(0xFF)  # what a workspace held before does not matter
        graph.replay()
        torch.cuda.synchronize()
        e = D.dora_muon(*up, 0.02, params_out=p2(up[0]), momenta_out=p2(up[2]))
        for i in range(3):
            assert torch.equal(po[i], e[0][i]) and torch.equal(mo[i], e[1][i])
        assert torch.equal(O, D.dora_orthogonalize(up[1][2]))


def test_python_refuses():
    A, g, m = (torch.zeros(8, 64, device=DEV, dtype=t) for t in (BF, BF, F32))
    for bad, call in (
            (ValueError, lambda: D.dora_orthogonalize(A[0])),
            (TypeError, lambda: D.dora_orthogonalize(A.half())),
            (ValueError, lambda: D.dora_orthogonalize(A[:, ::2])),
            (ValueError, lambda: D.dora_orthogonalize(A.cpu())),
            (D.DoraError, lambda: D.dora_orthogonalize(A, steps=0)),
            (D.DoraError, lambda: D.dora_orthogonalize(A, steps=17)),
            (D.DoraError, lambda: D.dora_orthogonalize(A, eps=-1.0)),
            (D.DoraError, lambda: D.dora_orthogonalize(A, coefficients=(1.0, float("nan"), 0.0))),
            (ValueError, lambda: D.dora_orthogonalize(A, coefficients=(1.0, 2.0))),
            (D.DoraError, lambda: D.dora_orthogonalize(A, ws=torch.empty(64, dtype=torch.uint8,
                                                                          device=DEV))),
            (ValueError, lambda: D.dora_muon([A], [g], [], 0.1)),
            (TypeError, lambda: D.dora_muon([A], [g], [g], 0.1)),
            (TypeError, lambda: D.dora_muon([A], [m], [m], 0.1)),
            (ValueError, lambda: D.dora_muon([A], [g[:4].contiguous()], [m], 0.1)),
            (ValueError, lambda: D.dora_muon([A], [g], [m], 0.1, scales=[1.0, 2.0])),
            (D.DoraError, lambda: D.dora_muon([A, A], [g, g], [m, m.clone()], 0.1)),
            (D.DoraError, lambda: D.dora_muon([A], [A], [m], 0.1)),
            (D.DoraError, lambda: D.dora_muon([A], [g], [m], float("nan")))):
        with pytest.raises(bad):
            call()
    assert D.dora_muon([], [], [], 0.1) == ([], [])
