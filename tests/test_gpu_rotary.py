"""GPU parity of rotary positions against the fp64 oracle.

Tolerance: the angle's part of a turn is rounded to 2^-26 turns and formed from 64-bit products that are off by at
most |p freq| 2^-52 radians (below 2^-25 here); sine and cosine are within 2^-23 of it; scale, two products and a
sum round four times.  2^-21 |scale| (|u| + |v|) covers them; the output's half step comes on top.
"""
import numpy as np
import pytest
import torch

import oracle as O
from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


def check(got, x, freq, pos, dtype, interleaved, scale=1.0, inverse=False):
    """got, x: [B,H,T,D] tensors."""
    ref = O.rotary(f64(x), f64(freq), pos, interleaved, scale, inverse)
    R = 2 * len(freq)
    size = np.zeros(ref.shape)
    a = np.abs(f64(x))
    if interleaved:
        size[..., 0:R:2] = size[..., 1:R:2] = a[..., 0:R:2] + a[..., 1:R:2]
    else:
        size[..., :R // 2] = size[..., R // 2:R] = a[..., :R // 2] + a[..., R // 2:R]
    tol = 2.0 ** -21 * abs(scale) * size
    allowed = tol + HALF[dtype] * (np.abs(ref) + tol)
    bad = ~(np.abs(f64(got) - ref) <= allowed)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"
    assert np.array_equal(f64(got)[..., R:], f64(x)[..., R:])


SHAPES = [  # B, Hq, Hk, T, D, R
    (1, 1, 0, 1, 2, 2), (2, 4, 4, 1, 64, 64), (1, 8, 2, 33, 128, 64), (3, 5, 1, 50, 90, 50), (2, 3, 3, 17, 96, 96),
    (2, 2, 1, 40, 256, 256), (1, 1, 1, 9, 7, 6), (1, 2, 2, 5, 1024, 512), (1, 16, 16, 300, 64, 32), (2, 1, 1, 6, 36, 12),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout,out_layout", [("bhtd", "bhtd"), ("bthd", "bhtd"), ("bhtd", "bthd"), ("bthd", "bthd")])
@pytest.mark.parametrize("B,Hq,Hk,T,D,R", SHAPES)
def test_rotary_against_oracle(B, Hq, Hk, T, D, R, dtype, interleaved, layout, out_layout):
    gen = torch.Generator().manual_seed(D + T)
    freq, _ = gla.rotary_frequencies(R)
    pos = torch.randint(0, 1 << 20, (B, T), generator=gen)
    x = {"q": torch.randn(B, Hq, T, D, generator=gen).to(dtype)}
    x["k"] = torch.randn(B, Hk, T, D, generator=gen).to(dtype) if Hk else None
    turn = lambda t, lay: t if t is None or lay == "bhtd" else t.transpose(1, 2).contiguous()  # noqa: E731
    put = {n: None if t is None else turn(t, layout).cuda() for n, t in x.items()}
    how = dict(pos=pos.cuda(), interleaved=interleaved, layout=layout, out_layout=out_layout)
    got = dict(zip(("q", "k"), gla.rotary(put["q"], put["k"], freq, **how)))
    for n in ("q", "k"):
        if x[n] is None:
            assert got[n] is None
            continue
        check(turn(got[n], out_layout), x[n], freq, pos, dtype, interleaved)
    # the backward takes gradients in the outputs' layout and returns them in the inputs'
    grads = {n: None if t is None else turn(t, out_layout).cuda() for n, t in x.items()}
    back = dict(zip(("q", "k"), gla.rotary_bwd(grads["q"], grads["k"], freq, **how)))
    for n in ("q", "k"):
        if x[n] is not None:
            assert back[n].shape == put[n].shape
            check(turn(back[n], layout), x[n], freq, pos, dtype, interleaved, inverse=True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_positions(interleaved):
    """Counted from an offset, shared by the batch, one row each, far out, and below zero."""
    B, H, T, D = 3, 2, 21, 64
    freq, scale = gla.rotary_frequencies(D, scaling="yarn", factor=16.0, trained=4096)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(B, H, T, D, generator=gen)
    q = x.cuda()
    count = np.arange(T)[None].repeat(B, 0)
    far = 100_000_000
    for pos, pos0, want in ((None, 0, count), (None, far, count + far), (torch.arange(T), 5, count + 5),
                            (torch.arange(T).repeat(B, 1) - 9, 0, count - 9)):
        got, none = gla.rotary(q, None, freq, pos=None if pos is None else pos.cuda(), pos0=pos0, interleaved=interleaved,
                               scale=scale)
        assert none is None
        check(got, x, freq, want, F32, interleaved, scale)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_many_heads_share_their_sines(interleaved):
    """Enough tokens that a thread turns several heads, across the border of q and k."""
    B, Hq, Hk, T, D = 2, 7, 3, 4099, 64
    gen = torch.Generator().manual_seed(2)
    q, k = torch.randn(B, Hq, T, D, generator=gen).to(BF16), torch.randn(B, Hk, T, D, generator=gen).to(BF16)
    freq, _ = gla.rotary_frequencies(48)
    qo, ko = gla.rotary(q.cuda(), k.cuda(), freq, interleaved=interleaved)
    pos = np.arange(T)[None].repeat(B, 0)
    check(qo, q, freq, pos, BF16, interleaved)
    check(ko, k, freq, pos, BF16, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_and_unaligned(interleaved):
    import ctypes
    B, H, T, D, R = 2, 3, 37, 64, 32
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(B, H, T, D, generator=gen).to(BF16)
    freq, _ = gla.rotary_frequencies(R)
    want, _ = gla.rotary(x.cuda(), None, freq, interleaved=interleaved)
    for shift in (0, 1, 2, 4):
        pad = 16
        flat = torch.full((x.numel() + 2 * pad + shift,), 3.0, dtype=BF16, device="cuda")
        q = flat[pad + shift:pad + shift + x.numel()]
        q.copy_(x.reshape(-1))
        code = gla.load_library().gla_rotary(
            q.data_ptr(), None, q.data_ptr(), None, freq.data_ptr(), None, 0, 0, B, H, 0, T, D, R, 1.0, int(interleaved), 0, 0, 0,
            1, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert code == 0
        torch.cuda.synchronize()
        assert torch.equal(q.view(x.shape), want)
        assert torch.all(flat[:pad + shift] == 3) and torch.all(flat[pad + shift + x.numel():] == 3)


def test_rotary_captured():
    B, H, T, D = 2, 4, 64, 128
    freq, _ = gla.rotary_frequencies(D)
    q, k = torch.randn(B, H, T, D, device="cuda", dtype=BF16), torch.randn(B, H, T, D, device="cuda", dtype=BF16)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    gla.rotary(q, k, freq, pos=pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = gla.rotary(q, k, freq, pos=pos)
    pos.copy_(torch.arange(T) + 1000)  # positions are read at replay
    graph.replay()
    torch.cuda.synchronize()
    want = gla.rotary(q, k, freq, pos0=1000)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_rotary_empty_and_binding_refusals():
    freq, _ = gla.rotary_frequencies(16)
    e = torch.empty(2, 3, 0, 16, device="cuda")
    assert gla.rotary(e, e, freq)[0].shape == (2, 3, 0, 16)
    q = torch.zeros(2, 3, 5, 16, device="cuda")
    with pytest.raises(gla.GLAError, match="freq must be"):
        gla.rotary(q, q, freq.float())
    with pytest.raises(gla.GLAError, match="freq"):
        gla.rotary(q, q, freq[None])
    with pytest.raises(gla.GLAError):
        gla.rotary(q, q, torch.ones(9, dtype=torch.float64, device="cuda"))  # R = 18 > D
    with pytest.raises(gla.GLAError, match="pos must be"):
        gla.rotary(q, q, freq, pos=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(gla.GLAError, match="pos must be"):
        gla.rotary(q, q, freq, pos=torch.zeros(1, 5, dtype=torch.int64, device="cuda"))
    with pytest.raises(gla.GLAError, match="k must be"):
        gla.rotary(q, q.to(BF16), freq)
    with pytest.raises(gla.GLAError, match="k must be"):
        gla.rotary(q, q[:, :, :4], freq)
    with pytest.raises(gla.GLAError, match="layout"):
        gla.rotary(q, q, freq, layout="tbhd")
