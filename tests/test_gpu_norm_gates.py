"""The norm's fp32 activations by themselves, against 64 bits: with w = 0 and b = 1 the normalised value is exactly 1,
so y = act(z), and with dy = 1 the gate's gradient is the activation's slope."""
import numpy as np
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu


def silu(v):
    return v / (1 + np.exp(-v))


def sigmoid(v):
    return 1 / (1 + np.exp(-v))


# e^-v is off by 2^-22 (the base-2 exponential) and 2^-23 (the correction of its argument and the product with it), the
# sum with 1 by 2^-24, the reciprocal by 2^-23: 2^-21 for the sigmoid however far v lies, and 2^-24 more for the product.
@pytest.mark.parametrize("lo,hi", [(-80.0, -10.0), (-10.0, 10.5), (10.0, 80.0)])
@pytest.mark.parametrize("act,of", [("silu", silu), ("sigmoid", sigmoid)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("D", [512, 514, 517])
def test_activation_of_far_values(lo, hi, act, of, gate, D):
    v = torch.linspace(lo, hi, D, dtype=torch.float64).to(torch.float32).view(1, 1, 1, D)
    x = torch.randn(1, 1, 1, D, generator=torch.Generator().manual_seed(1)).cuda()
    w, z, b = torch.zeros(1, D), (v if gate else None), (torch.ones(1, D) if gate else v.view(1, D))
    y = gla.group_norm_fwd(x, z.cuda() if gate else None, w.cuda(), b.cuda(), kind="rms", act=act, layout="bthd")
    ref = of(f64(v))
    assert np.max(np.abs(f64(y) - ref) / np.abs(ref)) <= 2.0 ** -20.5


# The slope of the SiLU is s (1 + v (1 - s)): its terms' sizes are s and |v| s (1 - s); each is off by 2^-21 for s, 2^-21 of
# s for 1 - s, and three roundings.
@pytest.mark.parametrize("lo,hi", [(-80.0, -10.0), (-10.0, 10.5)])
@pytest.mark.parametrize("D", [512, 514, 517])
def test_slope_of_far_gates(lo, hi, D):
    z = torch.linspace(lo, hi, D, dtype=torch.float64).to(torch.float32).view(1, 1, 1, D)
    x = torch.randn(1, 1, 1, D, generator=torch.Generator().manual_seed(1))
    w, b = torch.zeros(1, D), torch.ones(1, D)
    _, dz, _, _ = gla.group_norm_bwd(x.cuda(), torch.ones_like(x).cuda(), z.cuda(), w.cuda(), b.cuda(), kind="rms", act="silu",
                                     layout="bthd")
    v = f64(z)
    s = sigmoid(v)
    size = s * (1 + np.abs(v))
    assert np.max(np.abs(f64(dz) - s * (1 + v * (1 - s))) / size) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_at_the_ends_of_their_range(dtype, act):
    """Infinities, the type's largest values and NaN, each in its own channel."""
    most, inf = torch.finfo(dtype).max, float("inf")
    z = torch.tensor([inf, most, 1e30, 300.0, -300.0, -1e30, -most, float("nan")], dtype=dtype).view(1, 1, 1, 8)
    x = torch.ones_like(z)
    y = f64(gla.group_norm_fwd(x.cuda(), z.cuda(), torch.zeros(1, 8).cuda(), torch.ones(1, 8).cuda(), kind="rms", act=act,
                               layout="bthd")).reshape(8)
    up = f64(z).reshape(8)[:4] if act == "silu" else np.ones(4)
    assert np.array_equal(y[:4], up) and np.array_equal(y[4:7], np.zeros(3)) and np.isnan(y[7])
