"""GPU: orthogonalised matrices of low rank, one step to sixteen.

The gradient of a factor over few tokens has a lower rank than the factor.  The
directions that it lacks are multiplied by a at each step in Q, and the product
with U at the end takes them out again: what is rounded in between shows, as it
does in the steps as they are written.  The bound (low_rank_ref.py) has a share
for the n x n part and one for the product at the end; where both pass the size
of O itself (sixteen steps take 2^-24 of U to 24 times its size), O still has to
stay as bounded as the steps are."""
import pytest
import torch

from around_ref import half
from dora_adapter_amd import dora as D
from gpu_util import say
from low_rank_ref import COEFFICIENTS, QUINTIC, U, Steps, low_rank

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
STEPS = (1, 2, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16)


def ranks(n):
    return sorted({1, min(8, n), n // 4, n - 1})


def check(M, dt, steps=STEPS, coefficients=COEFFICIENTS):
    ref = Steps(M)
    X = M.to(DEV)
    for co in coefficients:
        for k in steps:
            O = D.dora_orthogonalize(X, steps=k, coefficients=co).cpu().double()
            want, bound = ref.run(k, co)
            size = float(torch.linalg.vector_norm(want))
            off = float(torch.linalg.vector_norm(O - want))
            assert torch.isfinite(O).all(), (k, co)
            assert off <= bound + size * half(dt), f"{k} steps {co}: off by {off:.3e}, bound {bound:.3e}"
            # (1.21 is the most that the quintic makes of a singular value; the rest is room for
            # the product at the end where Q has 2^25: 2^-24 of that)
            assert float(torch.linalg.matrix_norm(O, 2)) <= 1.21 + 4, (k, co)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,length", [(16, 333), (64, 1000), (128, 700), (384, 600)])
def test_whole_numbers(n, length, dt):
    """Exactly of that rank."""
    for rank in ranks(n):
        say("low rank", n, length, rank, dt)
        check(low_rank(n + rank, n, length, rank, dt), dt)
        check(low_rank(n + rank, length, n, rank, dt), dt, steps=(5, 8, 16))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,length", [(16, 4096), (64, 1000), (130, 700), (384, 600)])
def test_rounded_products(n, length, dt):
    """Of that rank but for the elements' rounding, whose directions the steps bring up."""
    for rank in ranks(n):
        say("low rank, rounded", n, length, rank, dt)
        check(low_rank(n + rank, n, length, rank, dt, whole=False), dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", [(48, 900), (900, 48), (200, 640), (640, 200)])
def test_singular_values_far_apart(shape, dt):
    """Full rank, singular values from 1 to 1e-4, and rows far smaller than others."""
    g = torch.Generator().manual_seed(5)
    n, length = min(shape), max(shape)
    left = torch.linalg.qr(torch.randn(n, n, generator=g, dtype=torch.float64))[0]
    right = torch.linalg.qr(torch.randn(length, n, generator=g, dtype=torch.float64))[0]
    M = left @ torch.diag(torch.logspace(0, -4, n, dtype=torch.float64)) @ right.T
    graded = low_rank(3, n, length, n // 4, F32, whole=False).double() \
        * torch.exp2(-20 * torch.rand(n, 1, generator=g).double())
    for m in (M, graded):
        say("singular values far apart", shape, dt)
        check((m if shape[0] == n else m.T).to(dt).contiguous(), dt, steps=(3, 5, 8, 12, 16),
              coefficients=(QUINTIC,))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,length", [(5, 70000), (48, 9000), (64, 64), (256, 256), (700, 1500)])
def test_sixteen_steps_stay_bounded(n, length, dt):
    """No rounding of G leaves an eigenvalue that the last steps take out of their range."""
    for rank in {1, max(n // 3, 1)}:
        for whole in (True, False):
            say("sixteen steps", n, length, rank, dt, whole)
            M = low_rank(rank, n, length, rank, dt, whole)
            for co in COEFFICIENTS:
                for m in (M, M.T.contiguous()):
                    O = D.dora_orthogonalize(m.to(DEV), steps=16, coefficients=co).cpu().double()
                    assert torch.isfinite(O).all() and float(torch.linalg.matrix_norm(O, 2)) <= 1.21 + 4


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("steps", [5, 8])
def test_updates_of_low_rank(steps, dt):
    """dora_muon's step: momenta of low rank, parameters of zeros, so that they come out as O."""
    shapes = [(16, 500), (64, 900), (900, 64), (384, 512), (512, 384)] * 2
    g = torch.Generator().manual_seed(7)
    grads = [low_rank(k, *s, (1, 4, 16)[k % 3], dt) for k, s in enumerate(shapes)]
    momenta = [low_rank(50 + k, *s, (1, 4, 16)[k % 3], F32) * 0.37 for k, s in enumerate(shapes)]
    say("muon of low rank", steps, dt)
    zeros = [torch.zeros(*s, dtype=dt, device=DEV) for s in shapes]
    out, new = D.dora_muon(zeros, [t.to(DEV) for t in grads], [t.to(DEV) for t in momenta], 1.0,
                           scales=[-1.0] * len(shapes), steps=steps, mu=0.75)
    for k, (gr, m) in enumerate(zip(grads, momenta)):
        m1 = 0.75 * m.double() + gr.double()
        V = gr.double() + 0.75 * m1
        ref = Steps(V)
        want, bound = ref.run(steps, QUINTIC)
        # U is a few fp32 roundings of its terms off, and moves O by at most as the steepest
        # singular value does
        terms = gr.double().abs() + 2 * (0.75 * m1).abs() + 2 * (0.75 * m.double()).abs()
        moved = 3 * U * float(torch.linalg.vector_norm(terms) / torch.linalg.vector_norm(V))
        bound += ref.steepest(steps, QUINTIC) * moved + float(torch.linalg.vector_norm(want)) * half(dt)
        off = float(torch.linalg.vector_norm(out[k].cpu().double() - want))
        assert off <= bound, f"matrix {k} {tuple(gr.shape)}: off by {off:.3e}, bound {bound:.3e}"
