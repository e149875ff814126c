"""The scan, the norm and rotary over tensors of more than 2^31 values: the same block of tokens again and again.

Every repetition has to give the bits of the first one, and the first one is compared with the oracle.  In one long
sequence each repetition of the scan starts with a reset (g = -inf), which nothing passes, forward or backward.
"""
import pytest
import torch

import test_gpu_group_norm as N
import test_gpu_rotary as R
import test_gpu_scan as S
from chunkwise_linear_rnn_02_b200 import binding as gla

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def many(t, n, dim=0):
    return torch.cat([t.cuda()] * n, dim)


def same(big, n, dim=0):
    """The first of n equal parts along dim, after a look that the others are equal to it."""
    parts = big.chunk(n, dim)
    assert len(parts) == n and parts[0].shape[dim] * n == big.shape[dim]
    view = big.unflatten(dim, (n, -1))
    assert bool((view == view.narrow(dim, 0, 1)).all())
    return parts[0].cpu()


@pytest.mark.parametrize("D", [1024, 1001])
@pytest.mark.parametrize("long", [False, True])
def test_scan_over_2_31_values(D, long):
    T = 2048
    n = 2 ** 31 // (T * D) + 2
    d = S.make(1, 1, T, D, BF16, seed=D)
    d["g"][:, :, 0] = -float("inf")
    dim = 2 if long else 0
    g, x, do = (many(d[k], n, dim) for k in ("g", "x", "do"))
    assert g.numel() > 2 ** 31
    o, _, hc = gla.scan_fwd(g, x, save_states=True)
    dg, dx, _ = gla.scan_bwd(g, x, do, hc=hc)
    got = {"o": same(o, n, dim), "dg": same(dg, n, dim), "dx": same(dx, n, dim)}
    ref, tol = S.bounds(d, False, False, False)
    for k, v in got.items():
        S.check(k, v, ref[k], tol[k], BF16)
    assert gla.device_error() == 0


@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_norm_over_2_31_values(layout):
    H, T, D = 4, 64, 512
    n = 2 ** 31 // (H * T * D) + 2
    d = N.make(1, H, T, D, BF16, H, True, layout, seed=8)
    how = dict(kind="group", act="silu", eps=1e-3, layout=layout)
    x, z, dy = (many(d[k], n) for k in ("x", "z", "dy"))
    w, b = d["w"].cuda(), d["b"].cuda()
    y = gla.group_norm_fwd(x, z, w, b, **how)
    dx, dz, _, _ = gla.group_norm_bwd(x, dy, z, w, b, **how)
    c = N.cuda(d)
    assert torch.equal(same(y, n), gla.group_norm_fwd(c["x"], c["z"], w, b, **how).cpu())
    few = gla.group_norm_bwd(c["x"], c["dy"], c["z"], w, b, **how)
    assert torch.equal(same(dx, n), few[0].cpu()) and torch.equal(same(dz, n), few[1].cpu())
    N.check_all(d, how, BF16)


@pytest.mark.parametrize("layout,out_layout", [("bthd", "bhtd"), ("bhtd", "bthd")])
def test_rotary_over_2_31_values(layout, out_layout):
    H, T, D = 16, 64, 128
    n = 2 ** 31 // (H * T * D) + 2
    freq, _ = gla.rotary_frequencies(D)
    q = torch.randn(1, H, T, D, generator=torch.Generator().manual_seed(9)).to(BF16)
    turn = lambda t, lay: t if lay == "bhtd" else t.transpose(1, 2).contiguous()  # noqa: E731
    out, _ = gla.rotary(many(turn(q, layout), n), None, freq, layout=layout, out_layout=out_layout)
    R.check(turn(same(out, n), out_layout), q, freq, torch.arange(T).expand(1, T), BF16, False)
