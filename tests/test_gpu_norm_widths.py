"""GPU parity of every variant of the group norm, with the bounds of test_gpu_group_norm.py: widths that 16-byte vectors do not
divide, widths that fill no variant, few tokens and enough for several steps a block, and tensors off their alignment."""
import ctypes

import pytest
import torch

import oracle as O
import test_gpu_group_norm as N
from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HOWS = [("group", "silu", True, True, "bhtd"), ("rms", "sigmoid", True, False, "bthd"), ("group", "silu", False, False, "bthd"),
        ("rms", "none", False, True, "bhtd"), ("group", "none", True, True, "bhtd"), ("rms", "sigmoid", False, False, "bhtd")]


# Even widths off 16 bytes go by two values (up to 64, 256, 1,024 and beyond), odd ones by one; the rest by 16 bytes.
# 2 * 2 * 5 rows are one step a block; the longer ones several.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [2, 50, 62, 66, 254, 258, 300, 1002, 1026, 2050, 8190,
                               3, 33, 63, 65, 99, 255, 257, 999, 1025, 2049, 8191,
                               8, 80, 192, 320, 384, 768, 1280, 2560, 5120])
@pytest.mark.parametrize("kind,act,gate,per_head,layout", HOWS)
def test_widths(dtype, D, kind, act, gate, per_head, layout):
    how = dict(kind=kind, act=act, eps=1e-3, layout=layout)
    N.check_all(N.make(2, 2, 5, D, dtype, 2 if per_head else 1, gate, layout, seed=D), how, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,T", [(50, 1500), (300, 1500), (1002, 1500), (2050, 400), (63, 1500), (99, 1500), (257, 1500), (1025, 400),
                                 (80, 6000), (320, 1500), (768, 1500), (2560, 400), (5120, 300)])
@pytest.mark.parametrize("kind,act,gate,per_head,layout", HOWS[:3])
def test_widths_over_several_steps(dtype, D, T, kind, act, gate, per_head, layout):
    how = dict(kind=kind, act=act, eps=1e-3, layout=layout)
    N.check_all(N.make(2, 2, T, D, dtype, 2 if per_head else 1, gate, layout, seed=D + T), how, dtype)


# One tensor at a time starts one, two or four values behind its alignment, between words that have to stay as they are.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("moved", ["x", "z", "y", "dy", "dx", "dz", "all"])
@pytest.mark.parametrize("D", [64, 80])
def test_tensors_off_their_alignment(dtype, shift, moved, D):
    B, H, T, pad = 2, 3, 37, 32
    how = dict(kind="group", act="silu", eps=1e-3, layout="bhtd")
    d = N.make(B, H, T, D, dtype, H, True, "bhtd", seed=D)
    lib, code, n = gla.load_library(), gla.DTYPE_CODE[dtype], B * H * T * D
    buf = {}
    for k in ("x", "z", "y", "dy", "dx", "dz"):
        at = pad + (shift if moved in (k, "all") else 0)
        whole = torch.full((n + 2 * pad + shift,), 7.0, dtype=dtype, device="cuda")
        buf[k] = (whole, whole[at:at + n])
        if k in d:
            buf[k][1].copy_(d[k].reshape(-1))
    w, b = d["w"].cuda(), d["b"].cuda()
    dw, db = torch.empty_like(w), torch.empty_like(b)
    p = {k: v[1].data_ptr() for k, v in buf.items()}
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.gla_group_norm_fwd(p["x"], p["z"], w.data_ptr(), b.data_ptr(), p["y"], B, H, T, D, H, 0, 1, 1e-3, 0, code, st) == 0
    need = lib.gla_group_norm_bwd_workspace(B, H, T, D, H, 1, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.gla_group_norm_bwd(p["x"], p["z"], w.data_ptr(), b.data_ptr(), p["dy"], p["dx"], p["dz"], dw.data_ptr(), db.data_ptr(),
                                  B, H, T, D, H, 0, 1, 1e-3, 0, code, ws.data_ptr(), need, st) == 0
    torch.cuda.synchronize()
    for whole, inner in buf.values():
        at = (inner.data_ptr() - whole.data_ptr()) // whole.element_size()
        assert torch.all(whole[:at] == 7) and torch.all(whole[at + n:] == 7)
    a = {k: f64(v) for k, v in d.items()}
    size = N.sizes(d, how)
    N.check("y", buf["y"][1].view(B, T, H, D), O.group_norm_fwd(a["x"], a["z"], a["w"], a["b"], **how), size["y"], dtype)
    ref = O.group_norm_bwd(a["x"], a["dy"], a["z"], a["w"], a["b"], **how)
    rows = B * H * T
    for k, got, r in zip(("dx", "dz", "dw", "db"), (buf["dx"][1].view(B, H, T, D), buf["dz"][1].view(B, T, H, D), dw, db), ref):
        wide = k in ("dw", "db")
        N.check(k, got, r, size[k], F32 if wide else dtype, N.K + (rows + 64) * 2.0 ** -24 if wide else N.K)
