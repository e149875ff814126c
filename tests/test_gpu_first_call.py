"""The scan, norm and rotary calls as the first thing a process does with the library, inside a stream capture: what
they set up on first use (kernel attributes, tensor maps) has to be legal there, and the replay gives what a plain
call gives."""
import subprocess
import sys
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys, torch
from chunkwise_linear_rnn_02_b200 import binding as gla
t = lambda *s, dtype=torch.bfloat16: torch.randn(s, device="cuda").to(dtype)
g, x, z = -t(1, 2, 3000, 64).abs() / 16, t(1, 2, 3000, 64), t(1, 3000, 2, 64)
w, S, freq = t(2, 64, dtype=torch.float32), t(1, 2, 64, dtype=torch.float32), gla.rotary_frequencies(64)[0]
g1, x1 = g[:, :, 0].contiguous(), x[:, :, 0].contiguous()
call = {
    "scan_fwd": lambda: gla.scan_fwd(g, x, save_states=True),
    "scan_bwd": lambda: gla.scan_bwd(g, x, x),
    "scan_step": lambda: (gla.scan_step(g1, x1, S.zero_()),),
    "group_norm_fwd": lambda: (gla.group_norm_fwd(x, z, w, w),),
    "group_norm_bwd": lambda: gla.group_norm_bwd(x, z, z, w, w),
    "rotary": lambda: gla.rotary(x, x, freq),
}[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
want = call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay differs"
assert gla.device_error() == 0
"""


@pytest.mark.parametrize("name", ["scan_fwd", "scan_bwd", "scan_step", "group_norm_fwd", "group_norm_bwd", "rotary"])
def test_first_call_is_captured(name):
    r = subprocess.run([sys.executable, "-c", PROGRAM, name], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
