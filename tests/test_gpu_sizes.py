"""Sizes at the ends of what the scan, the norm and rotary take: run, or refused by name."""
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_sizes_beyond_31_bits_are_refused():
    """Sizes go to the library as 32-bit ints: a longer axis is an error, not a shorter axis."""
    n = (1 << 32) + 8
    flat = torch.empty(n, dtype=BF16, device="cuda")
    t, wide = flat.view(1, 1, n, 1), flat.view(1, 1, 1, n)
    freq = torch.ones(1, dtype=torch.float64, device="cuda")
    two = flat.view(1, 1, n // 2, 2)
    calls = [lambda: gla.scan_fwd(t, t, output_final_state=False), lambda: gla.scan_fwd(wide, wide, output_final_state=False),
             lambda: gla.scan_bwd(t, t, t, need_dh0=False), lambda: gla.scan_step(wide[0], wide[0], torch.zeros(1, device="cuda")),
             lambda: gla.group_norm_fwd(t), lambda: gla.group_norm_bwd(t, flat.view(1, n, 1, 1)), lambda: gla.group_norm_fwd(wide),
             lambda: gla.rotary(two, None, freq), lambda: gla.rotary(two[:, :, :1], two.transpose(1, 2), freq)]
    for call in calls:
        with pytest.raises(gla.GLAError, match="2\\^31"):
            call()


def test_long_axes_of_empty_tensors_are_refused():
    """An empty sequence still has states: h0 of 2^32 + 1 heads is copied whole or not at all."""
    e = torch.empty(1, (1 << 32) + 1, 0, 1, dtype=BF16, device="cuda")
    with pytest.raises(gla.GLAError, match="2\\^31"):
        gla.scan_fwd(e, e)


def test_more_frequencies_than_channels_are_refused():
    """2^32 + 8 channels' frequencies would be 8 to the library: as many as a head of 8 has."""
    freq = torch.ones((1 << 31) + 4, dtype=torch.float64, device="cuda")
    with pytest.raises(gla.GLAError, match="freq must have at most"):
        gla.rotary(torch.zeros(1, 1, 1, 8, device="cuda"), None, freq)


@pytest.mark.parametrize("pos0", [1 << 63, -(1 << 63) - 1, 1 << 70])
def test_positions_beyond_64_bits_are_refused(pos0):
    q = torch.zeros(1, 1, 2, 4, device="cuda")
    with pytest.raises(gla.GLAError, match="pos0"):
        gla.rotary(q, None, torch.ones(2, dtype=torch.float64, device="cuda"), pos0=pos0)


@pytest.mark.parametrize("D", [(1 << 31) - 1, (1 << 31) - 16])
def test_scan_of_the_widest_rows(D):
    """One token of as many channels as the header allows: the last slab ends where 31 bits end."""
    x = torch.empty(1, 1, 1, D, dtype=BF16, device="cuda")
    x.view(-1)[:] = 1.0
    x.view(-1)[-100:] = torch.arange(100, device="cuda").to(BF16)
    g = torch.full_like(x, -1.0)
    o, _, hc = gla.scan_fwd(g, x, output_final_state=False, save_states=True)
    assert torch.equal(o, x)
    del o
    dg, dx, _ = gla.scan_bwd(g, x, x, hc=hc, need_dh0=False)
    assert torch.equal(dx, x) and not bool(dg.any())
    assert gla.device_error() == 0
