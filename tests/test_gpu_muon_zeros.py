"""GPU: a matrix of zeros has no direction: O is zeros whatever eps is, 0 too,
and an optimiser's step on a gradient and momentum of zeros (dA, while B is
still zeros) leaves the parameter but for its decay."""
import pytest
import torch

from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (30, 700), (700, 30), (700, 150), (150, 700)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-7])
def test_zeros(eps, dt):
    for shape in SHAPES:
        say("zeros", shape, eps, dt)
        for steps in (1, 5):
            O = D.dora_orthogonalize(torch.zeros(*shape, dtype=dt, device=DEV), eps=eps, steps=steps)
            assert torch.count_nonzero(O) == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-7])
def test_a_step_on_zeros_beside_another(eps, dt):
    g = torch.Generator().manual_seed(2)
    params = [torch.randn(*s, generator=g).to(dt).to(DEV) for s in SHAPES for _ in range(2)]
    grads = [torch.zeros_like(p) if k % 2 else torch.randn(*p.shape, generator=g).to(dt).to(DEV)
             for k, p in enumerate(params)]
    momenta = [torch.zeros(p.shape, device=DEV) for p in params]
    say("a step on zeros", eps, dt)
    out, new = D.dora_muon(params, grads, momenta, 0.5, weight_decay=0.5, eps=eps,
                           params_out=[torch.empty_like(p) for p in params],
                           momenta_out=[torch.empty_like(m) for m in momenta])
    for k, p in enumerate(params):
        assert torch.isfinite(out[k]).all(), k
        if k % 2:
            assert torch.count_nonzero(new[k]) == 0
            assert torch.equal(out[k], (0.75 * p.float()).to(dt))  # (one rounding of either)
        else:
            assert not torch.equal(out[k], (0.75 * p.float()).to(dt))
