"""CPU: the shapes of a block norm's gate: [d], or [G, d] with G dividing the
tokens (or one row for no tokens); any other is refused."""
import pytest
import torch

from dora_adapter_amd import dora as D


@pytest.mark.parametrize("shape,T,rows", [((7,), 6, 6), ((7,), 0, 1), ((1, 7), 6, 6), ((2, 7), 6, 3),
                                          ((6, 7), 6, 1), ((1, 7), 0, 1)])
def test_rows_a_gate(shape, T, rows):
    assert D._gate_rows(torch.ones(shape), T, 7) == rows
    assert D._gate_rows(None, T, 7) == 0


@pytest.mark.parametrize("shape,T", [((), 6), ((), 0), ((1, 5, 7), 0), ((1, 1, 7), 1), ((2, 3, 7), 6),
                                     ((0, 7), 0), ((0, 7), 6), ((4, 7), 6), ((12, 7), 6), ((2, 7), 0)])
def test_refused(shape, T):
    with pytest.raises(ValueError):
        D._gate_rows(torch.ones(shape), T, 7)
