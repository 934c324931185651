"""GPU: the scale of a 4-bit group for every fp32 significand of its largest
value, against integers: max / 6 at six significant bits, ties to even, decided
by the quotient itself.  (A product with 1 / 6 rounded to fp32 puts five
significands an octave on a tie that they lie below: 1.5703124, 1.6640624, ...)"""
import pytest
import torch

from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def six_bits_of_a_sixth(X):
    """s 2^8 for the scale s of X 2^-23, X from 2^23 to 2^24 - 1: X / 6 at six bits lies in [2^-3, 2^-2)
    times 2^23 in steps of 2^15, or from there on in steps of 2^16."""
    step = torch.where(2 * X < 3 * 2 ** 23, 1, 2)
    d = 6 * 2 ** 15 * step
    q, r = X // d, X % d
    return step * (q + ((2 * r > d) | ((2 * r == d) & (q % 2 == 1))).long())


@pytest.mark.parametrize("power", [0, -9, 100, -100])
def test_every_significand(power):
    say("scales of every significand", power)
    X = torch.arange(2 ** 23, 2 ** 24)
    x = (X.double() * 2.0 ** (power - 23)).float()
    x[::3] *= -1
    codes, scale = D.dora_quantize_fourbit(x[:, None].to(DEV), group=32)
    ref = six_bits_of_a_sixth(X).double() * 2.0 ** (power - 8)
    assert torch.equal(scale[:, 0].cpu().double(), ref)
    # the value itself is six scales, to half of a step of theirs
    values = D.dora_dequantize_fourbit(codes, scale, 1, group=32, dtype=torch.float32)
    assert torch.equal(values[:, 0].cpu().double(), torch.sign(x.double()) * 6 * ref)


def test_the_five_next_to_a_tie():
    """Below a tie by less than fp32's last place of the quotient: the smaller scale."""
    tops = [1.5703123807907104, 1.6640623807907104, 1.7578123807907104, 1.8515623807907104,
            1.9453123807907104]
    x = torch.tensor(tops)[:, None] * torch.tensor([1.0, -0.5, 0.25, 0.3])
    codes, scale = D.dora_quantize_fourbit(x.to(DEV), group=32)
    for top, s in zip(tops, scale[:, 0].cpu().double().tolist()):
        tie = round(top / 6 * 256) / 256  # (within 2^-24 of it, and above it)
        assert 0 < tie - top / 6 < 2.0 ** -24
        assert s == tie - 2.0 ** -8, (top, s)
