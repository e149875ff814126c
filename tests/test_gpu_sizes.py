"""The scan at the widest rows that it takes."""
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
