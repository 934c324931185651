"""GPU: matrices that share launches do not meet: what one holds changes no
other one's result, an infinity or a NaN included; and the singular values that
come out are those that the steps make."""
import pytest
import torch

import around_ref as R
from dora_adapter_amd import dora as D
from gpu_util import say
from low_rank_ref import QUINTIC, Steps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# shorter sides to 64 and past it, wide and tall, next to each other
SHAPES = [(48, 900), (260, 170), (900, 48), (130, 400), (48, 900), (400, 130), (64, 64), (9, 1)]


def problem(dt, seed=4):
    g = torch.Generator().manual_seed(seed)
    return [[torch.randn(*s, generator=g).to(t).to(DEV) * k for s in SHAPES]
            for t, k in ((dt, 1.0), (dt, 0.25), (F32, 0.5))]


def step(ps, gs, ms):
    return D.dora_muon(ps, gs, ms, 0.02, weight_decay=0.1, params_out=[torch.empty_like(p) for p in ps],
                       momenta_out=[torch.empty_like(m) for m in ms])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 2.0 ** 120])
def test_what_one_matrix_holds_stays_there(value, dt):
    ps, gs, ms = problem(dt)
    say("neighbours", value, dt)
    po, mo = step(ps, gs, ms)
    assert all(torch.isfinite(t).all() for t in po + mo)
    for k, shape in enumerate(SHAPES):
        changed = [t.clone() for t in gs]
        changed[k][shape[0] // 2, shape[1] // 2] = value
        po2, mo2 = step(ps, changed, ms)
        for i in range(len(SHAPES)):
            if i != k:
                assert torch.equal(po2[i], po[i]) and torch.equal(mo2[i], mo[i]), (k, i)
        if value < 2.0 ** 127 and value > 0:
            assert torch.isfinite(po2[k]).all()
        else:
            assert po2[k].isnan().all()
            bad = ~torch.isfinite(mo2[k])
            assert int(bad.sum()) == 1 and bad[shape[0] // 2, shape[1] // 2]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", [(96, 2048), (2048, 60)])
def test_singular_values_that_come_out(shape, dt):
    """Each is what the steps make of U's, to no more than O is off in all; from 2e-3 of the norm on
    between 0.67 and 1.21."""
    g = torch.Generator().manual_seed(3)
    k = min(shape)
    left, right = torch.randn(shape[0], k, generator=g), torch.randn(k, shape[1], generator=g)
    M = ((left * torch.arange(1, k + 1).float() ** -0.2) @ right).to(dt)
    say("singular values", shape, dt)
    O = D.dora_orthogonalize(M.to(DEV)).cpu().double()
    ref = Steps(M)
    want, bound = ref.run(5, QUINTIC)
    bound += float(torch.linalg.vector_norm(want)) * R.half(dt)
    s = torch.linalg.svdvals(O)
    assert float((s - torch.linalg.svdvals(want)).abs().max()) <= bound
    big = int((ref.s >= 2e-3).sum())
    assert big > k // 2 and int((s > 0.67 - bound).sum()) >= big and float(s.max()) < 1.21 + bound
