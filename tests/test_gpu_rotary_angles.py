"""The rotary angle's stated bound, |p freq| 2^-52 + |p| 2^-62 + 2^-30 radians: a pair (1, 0) turns to (cos A, sin A),
whose sine shows the angle where it is small."""
import numpy as np
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu


def sines(freq, p):
    """What a call makes of (1, 0) at position p: sin(p freq), fp32."""
    R = 2 * len(freq)
    q = torch.zeros(1, 1, 1, R, device="cuda")
    q[..., :R // 2] = 1
    return f64(gla.rotary(q, None, freq.cuda(), pos0=p)[0])[0, 0, 0, R // 2:]


# Below 1e-3 the sine is the angle to 2^-21 of it, and fp32 holds it to 2^-24 of it: 2^-22 of the angle covers the
# rotation's products beside that.
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("p", [1, 3, -1, -5])
def test_small_angles(p, sign):
    freq = sign * torch.logspace(-9, -4, 512, dtype=torch.float64)
    A = p * f64(freq)
    assert np.max(np.abs(sines(freq, p) - np.sin(A)) - 2.0 ** -22 * np.abs(A)) <= 2.0 ** -30 + 2.0 ** -52
    # and the rounding leans to neither side: over 512 angles the mean of errors of at most 2^-30 is below a fifth of that
    # (four standard deviations of a mean of uniform errors are 4 / sqrt(3 * 512) = 0.102 of the largest one)
    assert abs(np.mean(sines(freq, p) - np.sin(A))) <= 0.2 * 2.0 ** -30


# Far positions: the product's error is |p freq| 2^-52 + |p| 2^-62, the reference's angle is reduced exactly in integers.
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("p", [1 << 20, (1 << 31) + 7, 10 ** 12, -(10 ** 12)])
def test_far_positions(p, sign):
    from fractions import Fraction

    freq = sign * torch.logspace(-6, 1.2, 256, dtype=torch.float64)
    two_pi = Fraction(int("6283185307179586476925286766559005768394338798750"), 10 ** 48)
    ref = []
    for f in freq.tolist():
        A = Fraction(f) * p / two_pi
        ref.append(np.sin(2 * np.pi * float(A - round(A))))
    bound = np.abs(p * f64(freq)) * 2.0 ** -52 + abs(p) * 2.0 ** -62 + 2.0 ** -30
    assert np.all(np.abs(sines(freq, p) - np.array(ref)) <= bound + 2.0 ** -22)
