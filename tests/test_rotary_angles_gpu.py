"""Rotary angles at far positions on the GPU, against angles reduced exactly (rational arithmetic
with 80 digits of pi).

Turning (1, 0) and (0, 1) gives the sine and cosine themselves.  Tolerance: the angle is within
2 |pos| 2^-64 turns (the frequency as a 64-bit fraction of a turn), 2^-32 turns (its upper half) and
2^-28 turns (a float of up to an eighth of a turn), together 2.5e-8 radians beside the position's
share; the sine and cosine add one unit in the last place below 1, 2^-24.  9e-8 with both."""
import math
from fractions import Fraction

import pytest
import torch

from hybrid_softmax_linear_chunked_b200 import binding as rb

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089,
              10 ** 79)
POSITIONS = [0, 1, -1, 4095, (1 << 31) - 1, -(1 << 31), (1 << 40) + 123, -(1 << 40) - 77,
             (1 << 48) + 5, (1 << 50) + 7, -(1 << 52) + 1]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_softmax_linear_chunked_b200 import build
    build.build()
    rb.load()
    return torch.device("cuda", 0)


@pytest.mark.parametrize("D", [48, 44], ids=["vectors", "any"])  # both kernels
@pytest.mark.parametrize("inverse", [False, True])
def test_angles_of_far_positions(dev, D, inverse):
    freq, _ = rb.rotary_frequencies(32)
    freq[1:6] = torch.tensor([1.0, 0.7, -0.7, 3.0, 1e-9], dtype=torch.float64)
    n, half = len(POSITIONS), 16
    x = torch.zeros(1, 2, n, D, device=dev)
    x[0, 0, :, :half] = 1.0          # (1, 0) -> (cos, sin)
    x[0, 1, :, half:2 * half] = 1.0  # (0, 1) -> (-sin, cos)
    pos = torch.tensor([POSITIONS], dtype=torch.int64, device=dev)
    y = rb.rotary(x, None, freq.to(dev), positions=pos, inverse=inverse).cpu().double()
    for i, at in enumerate(POSITIONS):
        tol = 9e-8 + 2 * abs(at) * 2.0 ** -64 * 2 * math.pi
        for p in range(half):
            turns = Fraction(float(freq[p])) * at / (2 * PI)
            turns -= round(turns)
            a = 2 * math.pi * float(turns) * (-1 if inverse else 1)
            got = [float(z) for z in (y[0, 0, i, p], y[0, 0, i, half + p], y[0, 1, i, p],
                                      y[0, 1, i, half + p])]
            want = [math.cos(a), math.sin(a), -math.sin(a), math.cos(a)]
            off = max(abs(g - w) for g, w in zip(got, want))
            assert off <= tol, (at, float(freq[p]), off, tol)
