"""GPU parity of the group norm with an output gate, forward and backward, against the fp64 oracle.

Tolerances: with u32 = 2^-24, fp32 sums of D positive or mixed terms are off by at most (D/LANES + 12) u32 of the
sum of sizes, D/LANES <= 32 terms a lane, then a tree; the statistics, products and quotients add a dozen
roundings, the activations up to 2^-20 (approximate exponential and quotient at bf16).  K = 2^-18 of the sizes
of the terms that a result is summed from covers them; the outputs' own half step comes on top.  Weight
gradients add their rows one after another: (rows + 64) u32 of the sum of sizes, plus K.
"""
import numpy as np
import pytest
import torch

import oracle as O
from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu

K = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


def make(B, H, T, D, dtype, rows, gate, layout, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = r(B, H, T, D) * 2 + 0.5
    d = {"x": (x if layout == "bhtd" else x.transpose(1, 2).contiguous()).to(dtype), "dy": r(B, T, H, D).to(dtype)}
    d["z"] = (r(B, T, H, D) * 3).to(dtype) if gate else None
    d["w"], d["b"] = (1 + r(rows, D) / 4, r(rows, D) / 2) if rows else (None, None)
    return d


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def check(name, got, ref, size, dtype, k=K):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    allowed = k * size + HALF[dtype] * (np.abs(ref) + k * size) + 1e-37
    bad = ~(np.abs(got - ref) <= allowed)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, allowed {allowed[bad][0]:.2e}"


def sizes(d, how):
    """The sums of the sizes of the terms behind each result."""
    a = {k: None if v is None else f64(v) for k, v in d.items()}
    x = a["x"].transpose(0, 2, 1, 3) if how["layout"] == "bhtd" else a["x"]
    c = x - x.mean(-1, keepdims=True) if how["kind"] == "group" else x
    rstd = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + how["eps"])
    n = (np.abs(x) + (np.abs(x).mean(-1, keepdims=True) if how["kind"] == "group" else 0)) * rstd
    w = np.ones((1, x.shape[-1])) if a["w"] is None else np.abs(a["w"])
    u = n * w + (0 if a["b"] is None else np.abs(a["b"]))
    gate = a["z"] is not None
    v = np.abs(a["z"]) if gate else u
    act = {"none": v, "silu": v, "sigmoid": np.ones_like(v)}[how["act"]]     # bounds of |act|, |act'|, |act''|
    slope = {"none": 1.0, "silu": 1.1, "sigmoid": 0.25}[how["act"]] * np.ones_like(v)
    dy = np.abs(a["dy"])
    y = u * act if gate else u * slope + act
    du = dy * (act if gate else slope + u)       # without a gate act'(u) moves with u's error, |act''| <= 1
    dn = du * w
    dx = rstd * (dn + dn.mean(-1, keepdims=True) + n * (dn * n).mean(-1, keepdims=True)) * 2
    over = (0, 1) if w.shape[0] > 1 else (0, 1, 2)
    dw, db = (du * n).sum(over).reshape(w.shape), du.sum(over).reshape(w.shape)
    return {"y": y, "dz": dy * u * (slope + 1) if gate else None,
            "dx": dx.transpose(0, 2, 1, 3) if how["layout"] == "bhtd" else dx, "dw": dw, "db": db}


def check_all(d, how, dtype):
    a = {k: None if v is None else f64(v) for k, v in d.items()}
    c = cuda(d)
    size = sizes(d, how)
    y = gla.group_norm_fwd(c["x"], c["z"], c["w"], c["b"], **how)
    check("y", y, O.group_norm_fwd(a["x"], a["z"], a["w"], a["b"], **how), size["y"], dtype)
    got = gla.group_norm_bwd(c["x"], c["dy"], c["z"], c["w"], c["b"], **how)
    ref = O.group_norm_bwd(a["x"], a["dy"], a["z"], a["w"], a["b"], **how)
    rows = d["dy"].numel() // d["dy"].shape[-1]
    for n, g, r in zip(("dx", "dz", "dw", "db"), got, ref):
        if n == "dz" and d["z"] is None or n in ("dw", "db") and d["w"] is None:
            assert g is None
            continue
        wide = n in ("dw", "db")
        check(n, g, r, size[n], F32 if wide else dtype, K + (rows + 64) * 2.0 ** -24 if wide else K)
    return y, got


SHAPES = [
    (1, 1, 1, 1), (1, 3, 1, 8), (2, 4, 5, 64), (3, 2, 33, 128), (2, 5, 17, 256), (1, 4, 40, 512), (2, 3, 9, 130),
    (1, 2, 7, 72), (2, 1, 11, 1000), (1, 1, 6, 2048), (1, 2, 5, 333), (1, 1, 3, 4096), (1, 1, 3, 8192), (1, 1, 2, 8191),
    (2, 40, 300, 16), (1, 4, 3000, 96),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,D", SHAPES)
@pytest.mark.parametrize("kind,act,gate,per_head,layout", [
    ("group", "silu", True, True, "bhtd"), ("rms", "sigmoid", True, False, "bthd"), ("group", "silu", False, False, "bthd"),
    ("rms", "none", False, True, "bhtd"),
])
def test_norm_against_oracle(B, H, T, D, dtype, kind, act, gate, per_head, layout):
    how = dict(kind=kind, act=act, eps=1e-3, layout=layout)
    check_all(make(B, H, T, D, dtype, H if per_head else 1, gate, layout, seed=T * 7 + D), how, dtype)


@pytest.mark.parametrize("kind", ["group", "rms"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [True, False])
def test_norm_every_mode_without_weights(kind, act, gate):
    how = dict(kind=kind, act=act, eps=1e-5, layout="bhtd")
    check_all(make(2, 3, 19, 64, BF16, 0, gate, "bhtd", seed=3), how, BF16)


@pytest.mark.parametrize("kind", ["group", "rms"])
def test_norm_many_rows_of_a_warp(kind):
    """Rows of 1,024 values without a gate are one warp's; more of them than the GPU holds at once."""
    how = dict(kind=kind, act="silu", eps=1e-3, layout="bthd")
    check_all(make(1, 1, 6001, 1024, BF16, 1, False, "bthd", seed=11), how, BF16)


def test_norm_one_weight_alone():
    d = cuda(make(2, 3, 10, 64, F32, 3, True, "bhtd", seed=4))
    _, _, dw, db = gla.group_norm_bwd(d["x"], d["dy"], d["z"], d["w"], d["b"])
    only_w = gla.group_norm_bwd(d["x"], d["dy"], d["z"], d["w"], torch.zeros_like(d["b"]))
    assert gla.group_norm_bwd(d["x"], d["dy"], d["z"], w=d["w"])[3] is None
    assert torch.equal(gla.group_norm_bwd(d["x"], d["dy"], d["z"], w=d["w"])[2], only_w[2])
    assert gla.group_norm_bwd(d["x"], d["dy"], d["z"], b=d["b"])[2] is None
    assert torch.equal(gla.group_norm_bwd(d["x"], d["dy"], d["z"], b=d["b"])[3], db)  # db does not read w
    assert dw.shape == (3, 64)


def test_norm_far_from_zero_and_constant_rows():
    """A mean 1000 times the spread (the squares are summed after the mean is taken off: the centred values keep
    what fp32 subtraction leaves, 2^-24 of the mean a value), and rows without any spread (n = 0, y = act(z) b)."""
    how = dict(kind="group", act="silu", eps=1e-5, layout="bhtd")
    d = make(1, 2, 9, 128, F32, 2, True, "bhtd", seed=5)
    d["x"] = d["x"] + 2000
    check_all(d, how, F32)
    d["x"] = torch.full_like(d["x"], 3.25)
    c = cuda(d)
    y = gla.group_norm_fwd(c["x"], c["z"], c["w"], c["b"], **how)
    z = f64(d["z"])
    check("y", y, f64(d["b"]) * z / (1 + np.exp(-z)), np.abs(f64(d["b"]) * z), F32)
    assert torch.isfinite(gla.group_norm_bwd(c["x"], c["dy"], c["z"], c["w"], c["b"], **how)[0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_gates_far_out(dtype):
    """Gates at +-90 and +-1e4: the activation saturates without overflowing into NaN."""
    d = make(1, 1, 4, 32, dtype, 1, True, "bhtd", seed=6)
    d["z"][..., ::2] = 90.0
    d["z"][..., 1::4] = -90.0
    d["z"][..., 3::4] = -1e4
    for act in ("silu", "sigmoid"):
        how = dict(kind="rms", act=act, eps=1e-5, layout="bhtd")
        with np.errstate(over="ignore"):
            y, (dx, dz, dw, db) = check_all(d, how, dtype)
        for t in (y, dx, dz, dw, db):
            assert torch.isfinite(t).all()


def test_norm_infinite_values_stay_in_their_sums():
    """A gate that makes dw infinite: the last step's places without a row add nothing to the sums (an infinity there
    would turn into NaN), and other channels, rows and heads stay finite."""
    d = make(1, 2, 37, 64, F32, 2, True, "bhtd", seed=11)
    d["z"][0, 36, 1, 5] = float("inf")  # the last row of head 1
    d["dy"][0, 36, 1, 5] = 1.0
    d["x"][0, 1, 36, 5] = 7.0           # n > 0 there
    c = cuda(d)
    y = gla.group_norm_fwd(c["x"], c["z"], c["w"], c["b"])
    assert torch.isinf(y[0, 36, 1, 5]) and torch.isfinite(y[0, :36]).all() and torch.isfinite(y[:, :, 0]).all()
    dx, dz, dw, db = gla.group_norm_bwd(c["x"], c["dy"], c["z"], c["w"], c["b"])
    assert dw[1, 5] == float("inf") and db[1, 5] == float("inf")
    for t in (dw, db):
        t[1, 5] = 0
        assert torch.isfinite(t).all()
    assert torch.isfinite(dx[0, 0]).all() and torch.isfinite(dx[0, 1, :36]).all()


def test_norm_empty_and_unaligned():
    x = torch.empty(2, 3, 0, 16, device="cuda", dtype=BF16)
    w = torch.ones(3, 16, device="cuda")
    assert gla.group_norm_fwd(x, w=w).shape == (2, 0, 3, 16)
    dx, dz, dw, db = gla.group_norm_bwd(x, torch.empty(2, 0, 3, 16, device="cuda", dtype=BF16), w=w, b=w)
    assert dx.shape == x.shape and torch.all(dw == 0) and torch.all(db == 0)
    d = make(2, 2, 21, 64, BF16, 2, True, "bhtd", seed=7)
    c = cuda(d)
    want = gla.group_norm_fwd(c["x"], c["z"], c["w"], c["b"])
    for shift in (1, 2, 4):
        flat = torch.empty(d["x"].numel() + shift, dtype=BF16, device="cuda")
        flat[shift:] = c["x"].reshape(-1)
        got = gla.group_norm_fwd(flat[shift:].view(d["x"].shape), c["z"], c["w"], c["b"])
        torch.testing.assert_close(got.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -14)  # a bf16 step apart at most


def test_norm_repeats_bit_for_bit_in_graphs_and_streams():
    how = dict(kind="group", act="silu", layout="bhtd")
    d = cuda(make(4, 4, 500, 128, BF16, 4, True, "bhtd", seed=8))

    def step():
        return (gla.group_norm_fwd(d["x"], d["z"], d["w"], d["b"], **how),) + gla.group_norm_bwd(
            d["x"], d["dy"], d["z"], d["w"], d["b"], **how)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(out, want, other):
        assert torch.equal(a, b) and torch.equal(c, b)


def test_norm_binding_refusals():
    x = torch.zeros(1, 2, 8, 16, device="cuda", dtype=BF16)
    w = torch.zeros(2, 16, device="cuda")
    with pytest.raises(gla.GLAError, match="z must be"):
        gla.group_norm_fwd(x, z=x)  # [B,H,T,D] where [B,T,H,D] is wanted
    with pytest.raises(gla.GLAError, match="w and b must be"):
        gla.group_norm_fwd(x, w=torch.zeros(3, 16, device="cuda"))
    with pytest.raises(gla.GLAError, match="w and b must be"):
        gla.group_norm_fwd(x, w=torch.zeros(16, device="cuda"))
    with pytest.raises(gla.GLAError, match="w must be"):
        gla.group_norm_fwd(x, w=w.to(BF16))
    with pytest.raises(gla.GLAError, match="w must be"):
        gla.group_norm_fwd(x, w=w, b=w[:1])
    for bad in (dict(kind="batch"), dict(act="relu"), dict(layout="thd"), dict(eps=0.0)):
        with pytest.raises(gla.GLAError):
            gla.group_norm_fwd(x, **bad)
    with pytest.raises(gla.GLAError, match="dy must be"):
        gla.group_norm_bwd(x, x)
    with pytest.raises(gla.GLAError, match="contiguous"):
        gla.group_norm_fwd(x.transpose(1, 2), layout="bthd")
