"""How far the norm's weight gradients round: the blocks' partial rows are joined in pairs, not one after another."""
import numpy as np
import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [592, 1184])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_partial_rows_are_joined_in_pairs(dtype, T):
    """db of tokens that all carry the same positive gradients, a value for each channel: sums of equal terms, which an addition
    at a time rounds in one direction for long stretches.  Without a gate or an activation db is the plain sum of dy.
    A block adds its tokens one by one; the partial rows (as many as the workspace holds) go in 32 groups, eight joined in pairs
    (3 roundings) and added to the group's sum (one for each 256 rows), and the groups in pairs (5)."""
    D = 2048
    x = torch.randn(1, T, 1, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    c = (1 + torch.rand(D, generator=torch.Generator().manual_seed(2))).to(dtype)
    dy = c.expand(1, T, 1, D).contiguous().cuda()
    b = torch.zeros(1, D, device="cuda")
    db = gla.group_norm_bwd(x, dy, b=b, kind="rms", act="none", layout="bthd")[3]
    rows = gla.workspace_bytes("gla_group_norm_bwd", 1, 1, T, D, 1, 0, 1) // (4 * D)
    roundings = -(-T // rows) - 1 + -(-rows // 256) + 3 + 5
    ref = T * f64(c)
    assert np.max(np.abs(f64(db)[0] - ref) / ref) <= roundings * 2.0 ** -24
