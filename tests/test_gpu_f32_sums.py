"""GPU: an fp32 product's sums are chains of fmas in ascending K, bit for bit.

The chain is formed here with the C library's fmaf (correctly rounded), on operands
whose partial sums cancel, on denormal ones and on ordinary ones, for K that the
planner does not split."""
import ctypes
import ctypes.util

import numpy as np
import pytest
import torch

from dora_adapter_amd import dora as D
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

_libm = ctypes.CDLL(ctypes.util.find_library("m"))
_libm.fmaf.restype = ctypes.c_float
_libm.fmaf.argtypes = [ctypes.c_float] * 3


def chain(x, W, at):
    """sum_k x[i, k] W[j, k] for the pairs (i, j) of `at`, one fma a term."""
    out = []
    for i, j in at:
        c = 0.0
        for a, b in zip(x[i].tolist(), W[j].tolist()):
            c = _libm.fmaf(a, b, c)
        out.append(c)
    return np.array(out, dtype=np.float32)


def kinds(T, d_in, d_out, g):
    x, W = torch.randn(T, d_in, generator=g), torch.randn(d_out, d_in, generator=g)
    yield "ordinary", x, W
    # pairs of terms that nearly cancel, over twenty orders of magnitude
    big = torch.exp2(torch.randint(-30, 31, (d_in,), generator=g).float())
    xc, Wc = x * big, W.clone()
    xc[:, 1::2] = -xc[:, 0:d_in - d_in % 2:2] * (1 + 2.0 ** -20)
    Wc[:, 1::2] = Wc[:, 0:d_in - d_in % 2:2]
    yield "cancelling", xc, Wc
    # products and sums below 2^-126
    yield "denormal", x * 2.0 ** -70, W * 2.0 ** -62
    yield "denormal operands", x * 2.0 ** -130, W * 2.0 ** 10


@pytest.mark.parametrize("T,d_in,d_out", [(3, 5, 4), (7, 130, 9), (70, 333, 65), (64, 256, 128)])
def test_fp32_sums_are_fma_chains(T, d_in, d_out):
    g = torch.Generator().manual_seed(T + d_in)
    pick = np.random.default_rng(T)
    for kind, x, W in kinds(T, d_in, d_out, g):
        say("fp32 linear", T, d_in, d_out, kind)
        y = D.dora_linear(x.to(DEV), W.to(DEV)).cpu().numpy()
        at = [(0, 0), (T - 1, d_out - 1)] + [(int(pick.integers(T)), int(pick.integers(d_out)))
                                             for _ in range(60)]
        want = chain(x, W, at)
        got = np.array([y[i, j] for i, j in at], dtype=np.float32)
        assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), kind
