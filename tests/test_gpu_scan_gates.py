"""The scan's a = exp g and 1 - a, one factor at a time, against 64 bits.

One token with h0 = 0 gives b alone, one token backward gives a and 1 - a alone, so the bounds below hold them
without the slack that a state of many terms has.
"""
import numpy as np
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu

N = 4096


def span(lo, hi):
    """N gates from lo to hi, evenly spread, fp32."""
    return torch.linspace(lo, hi, N, dtype=torch.float64).to(torch.float32).view(1, 1, 1, N)


def ones(seed):
    """Values of either sign in [1, 2)."""
    gen = torch.Generator().manual_seed(seed)
    v = 1 + torch.rand(1, 1, 1, N, generator=gen)
    return torch.where(torch.rand(1, 1, 1, N, generator=gen) < 0.5, v, -v)


def relative(got, ref):
    return np.max(np.abs(f64(got) - ref) / np.abs(ref))


# g = n ln 2 + f, a = s + s p with s = 2^n and p = exp f - 1.  With u = 2^-24 (half a step of 1 at fp32): f is off by u / 2 in
# all, p by 2.4 u of itself (the polynomial 0.3, its sum's rounding 0.85, its earlier terms' 0.25, the product 1), and the products
# with s are exact.
#   1 - a  is -p for n = 0: 2.4 u.  For n = -1 it is 1/2 - p/2 >= 0.293: (0.207 * 2.4 u + 0.71 * u / 2) / 0.293 and the
#          sum's u, 3.9 u.  For smaller n it is 1 - a with more of the 1.  The product with x is u more: below 6 u.
#   a      0.41 * 2.4 u / 1.41 (or 0.3 * 2.4 u / 0.7), u / 2 from f, u from the sum, u from the product with what it
#          scales: 3.5 u, however strong the gate.
# bf16 gates: below 1/2 the polynomial is off by 1.5 u, the rest as above; from 1/2 on 1 - a has a's 4 u (the base-2
# exponential) and 1.25 |g| u (its argument) a / (1 - a) = 1.55 times or less, 7.2 u, and u / 2 / 0.39 of its own, and the product
# with x u: 9.5 u.
SHARE, FACTOR, SHARE_BF16 = 6 * 2.0 ** -24, 2.0 ** -22, 2.0 ** -20.7
RANGES = [(-0.01, -1e-4), (-0.125, -0.01), (-0.5, -0.125), (-4.0, -0.5), (-80.0, -4.0)]


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("form", ["sequence", "step", "backward"])
def test_share_of_the_complement(lo, hi, form):
    g, x = span(lo, hi), ones(1)
    ref = -np.expm1(f64(g)) * f64(x)
    c = [t.cuda() for t in (g, x)]
    if form == "sequence":
        got = gla.scan_fwd(*c, complement=True)[1]
        ref = ref[:, :, 0]
    elif form == "step":
        got = gla.scan_step(c[0][:, :, 0].contiguous(), c[1][:, :, 0].contiguous(), torch.zeros(1, 1, N, device="cuda"),
                            complement=True)
        ref = ref[:, :, 0]
    else:  # dx = (1 - a) d, with x in the place of dO
        got = gla.scan_bwd(c[0], torch.zeros_like(c[1]), c[1], complement=True)[1]
    assert relative(got, ref) <= SHARE


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("step", [False, True])
def test_share_of_the_complement_in_a_state_of_bf16_gates(lo, hi, step):
    """The state is fp32 whatever the type of the gates."""
    g, x = span(lo, hi).to(torch.bfloat16), ones(1).to(torch.bfloat16)
    ref = (-np.expm1(f64(g)) * f64(x))[:, :, 0]
    if step:
        got = torch.zeros(1, 1, N, device="cuda")
        gla.scan_step(g[:, :, 0].cuda(), x[:, :, 0].cuda(), got, complement=True)
    else:
        got = gla.scan_fwd(g.cuda(), x.cuda(), complement=True)[1]
    assert relative(got, ref) <= SHARE_BF16


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("form", ["sequence", "step", "backward"])
def test_strong_gates_keep_their_digits(lo, hi, complement, form):
    g, h = span(lo, hi), ones(2)
    ref = (np.exp(f64(g)) * f64(h))[:, :, 0]
    zero, row = torch.zeros_like(g).cuda(), h[:, :, 0].cuda()
    if form == "sequence":
        got = gla.scan_fwd(g.cuda(), zero, h0=row, complement=complement)[1]
    elif form == "step":
        got = gla.scan_step(g[:, :, 0].cuda(), zero[:, :, 0].contiguous(), row, complement=complement)
    else:
        got = gla.scan_bwd(g.cuda(), zero, h.cuda(), complement=complement)[2]
    assert relative(got, ref) <= FACTOR


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("complement", [False, True])
def test_gates_at_the_ends_of_their_range(dtype, complement):
    """-inf, the type's lowest value and gates whose exponential underflows forget everything; 0 and -0 keep everything;
    NaN stays NaN in its own channel."""
    low = torch.finfo(dtype).min
    g = torch.tensor([-float("inf"), low, -1e30, -1000.0, -104.0, 0.0, -0.0, float("nan")], dtype=dtype).view(1, 1, 1, 8).cuda()
    x, h = torch.full_like(g, 3.0), torch.full((1, 1, 8), 5.0, device="cuda")
    for o, S in ((gla.scan_fwd(g, x, h0=h, complement=complement)[:2]),
                 ((lambda s: (gla.scan_step(g[:, :, 0].contiguous(), x[:, :, 0].contiguous(), s, complement=complement), s))(h.clone()))):
        o, S = f64(o).reshape(8), f64(S).reshape(8)
        assert np.array_equal(o[:5], [3.0] * 5) and np.array_equal(S[:5], [3.0] * 5)
        assert np.array_equal(S[5:7], [5.0] * 2 if complement else [8.0] * 2) and np.isnan(S[7]) and np.isnan(o[7])
    dg, dx, dh0 = (f64(t).reshape(8) for t in gla.scan_bwd(g, x, torch.ones_like(x), h0=h, complement=complement))
    assert np.array_equal(dh0[:7], [0.0] * 5 + [1.0] * 2) and np.array_equal(dg[:5], [0.0] * 5)
    assert np.array_equal(dx[:7], [1.0] * 5 + ([0.0] * 2 if complement else [1.0] * 2))
    assert np.array_equal(dg[5:7], [2.0] * 2 if complement else [5.0] * 2) and np.isnan(dh0[7])
