"""The scan on tensors off their alignment: inputs, outputs and states start one, two or four values late, one at a time and
all at once, between words that have to stay as they are.  Any tensor of the sequence off 16 bytes (or off two values) takes the
whole call from TMA to copies by the threads, of two values or of one."""
import ctypes

import pytest
import torch

import test_gpu_scan as S
from chunkwise_linear_rnn_02_b200 import binding as gla

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("moved", ["g", "x", "do", "o", "dg", "dx", "h0", "dhT", "hc", "hT", "dh0", "all"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_tensors_off_their_alignment(dtype, complement, moved, shift):
    B, H, T, D, pad = 2, 2, 333, 72, 64
    d = S.make(B, H, T, D, dtype, seed=13, resets=0.002)
    ref, tol = S.bounds(d, complement, True, True)
    n, m, k = B * H * T * D, B * H * D, B * H * (-(-T // 64)) * D
    sizes = {"g": n, "x": n, "do": n, "o": n, "dg": n, "dx": n, "h0": m, "dhT": m, "hT": m, "dh0": m, "hc": k}
    buf = {}
    for name, size in sizes.items():
        at = pad + (shift if moved in (name, "all") else 0)
        whole = torch.full((size + 2 * pad + shift,), 7.0, dtype=F32 if size != n else dtype, device="cuda")
        buf[name] = (whole, whole[at:at + size])
        if name in d:
            buf[name][1].copy_(d[name].reshape(-1))
    lib, code, st = gla.load_library(), gla.DTYPE_CODE[dtype], ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = {name: inner.data_ptr() for name, (_, inner) in buf.items()}
    assert lib.gla_scan_fwd(p["g"], p["x"], p["h0"], p["o"], p["hT"], p["hc"], B, H, T, D, int(complement), code, st) == 0
    assert lib.gla_scan_bwd(p["g"], p["x"], None, p["hc"], p["do"], p["dhT"], p["dg"], p["dx"], p["dh0"], B, H, T, D, int(complement),
                            code, None, 0, st) == 0
    torch.cuda.synchronize()
    for name, (whole, inner) in buf.items():
        at = (inner.data_ptr() - whole.data_ptr()) // whole.element_size()
        assert torch.all(whole[:at] == 7) and torch.all(whole[at + sizes[name]:] == 7), name
    for name in ref:
        S.check(name, buf[name][1].view(ref[name].shape), ref[name], tol[name], F32 if name in ("hT", "dh0") else dtype)
    assert gla.device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_step_off_its_alignment(dtype, shift):
    B, H, D, pad = 3, 2, 77, 32
    d = S.make(B, H, 1, D, dtype, seed=14)
    ref, tol = S.bounds(d, True, True, False)
    n = B * H * D
    buf = {name: torch.full((n + 2 * pad + shift,), 7.0, dtype=F32 if name == "S" else dtype, device="cuda") for name in ("g", "x", "S", "o")}
    inner = {name: t[pad + shift:pad + shift + n] for name, t in buf.items()}
    for name, src in (("g", "g"), ("x", "x"), ("S", "h0")):
        inner[name].copy_(d[src].reshape(-1))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert gla.load_library().gla_scan_step(*(inner[name].data_ptr() for name in ("g", "x", "S", "o")), B, H, D, 1, gla.DTYPE_CODE[dtype],
                                            st) == 0
    torch.cuda.synchronize()
    for t in buf.values():
        assert torch.all(t[:pad + shift] == 7) and torch.all(t[pad + shift + n:] == 7)
    S.check("o", inner["o"].view(B, H, 1, D), ref["o"], tol["o"], dtype)
    S.check("S", inner["S"].view(B, H, D), ref["hT"], tol["hT"], F32)
