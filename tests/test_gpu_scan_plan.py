"""GPU parity of every kernel of the elementwise scan over many steps, with the bounds of test_gpu_scan.py: forward with kept
states, backward from them, resets and kept gates among the gates, and an odd number of tokens behind the last whole tile."""
import pytest
import torch

import test_gpu_scan as S
from chunkwise_linear_rnn_02_b200 import binding as gla
from scan_shapes import SHAPES

pytestmark = pytest.mark.gpu

CASES = [(t, s) for (t, _), shapes in SHAPES.items() for s in shapes]


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("dtype,shape", CASES, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_every_kernel_over_many_steps(dtype, shape, complement):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    B, T, D = shape
    d = S.make(B, 1, T, D, dtype, seed=T * 41 + D, resets=0.001, keeps=0.01)
    ref, tol = S.bounds(d, complement, True, True)
    got = S.run_all(d, complement)
    for n in ref:
        S.check(n, got[n], ref[n], tol[n], torch.float32 if n in ("hT", "dh0") else dtype)
    assert gla.device_error() == 0
