"""GPU: matrices far below eps, or norms and eps far from one: U / (|U| + eps)
leaves fp32's range long before O does, and neither U nor Q may lose bits there.

The bound is that of low_rank_ref.py, its share of the output's rounding, and
nothing absolute: the results are far below one."""
import pytest
import torch

from around_ref import half
from dora_adapter_amd import dora as D
from gpu_util import say
from low_rank_ref import QUINTIC, Steps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("power,eps", [(-128, 1e-7), (-120, 1e-7), (-112, 1e-7), (-100, 1e-7), (-80, 1e-7),
                                       (-60, 1e-7), (-110, 1e-20), (-128, 1e-30), (0, 2.0 ** 100),
                                       (-20, 2.0 ** 90), (100, 2.0 ** 127), (110, 1e-7), (60, 2.0 ** 60)])
def test_far_from_eps(power, eps, dt):
    for shape in ((30, 700), (700, 30), (150, 700), (700, 150)):
        g = torch.Generator().manual_seed(5)
        M = (torch.randn(*shape, generator=g).to(dt).double() * 2.0 ** power).to(dt)
        say("far from eps", shape, power, eps, dt)
        ref = Steps(M, eps)
        want, bound = ref.run(5, QUINTIC, least=0.0)
        O = D.dora_orthogonalize(M.to(DEV), eps=eps).cpu().double()
        size = float(torch.linalg.vector_norm(want))
        off = float(torch.linalg.vector_norm(O - want))
        assert off <= bound + size * half(dt), f"{shape}: off by {off / size:.3e} of {size:.3e}"
