"""Pins of the fp64 oracle of the operators around the recurrences (CPU): the scan against GLA with
1 x 1 states and against its unrolled sum, the reverse modes against central differences, rotary
against complex multiplication and its own inverse; and the frequencies the binding makes."""
import numpy as np
import pytest
import torch

import oracle as O
from chunkwise_linear_rnn_02_b200 import binding as gla


def _diff(f, x, dy, eps=1e-6):
    """Central differences of sum(dy * f(x)) by every element of x."""
    d = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + eps
        hi = f()
        x[i] = keep - eps
        lo = f()
        x[i] = keep
        d[i] = sum(float((w * (h - l)).sum()) for w, h, l in zip(dy, hi, lo)) / (2 * eps)
    return d


@pytest.mark.parametrize("complement", [False, True])
def test_scan_is_gla_with_one_by_one_states(rng, complement):
    B, H, T, D = 2, 3, 9, 4
    g, x = -rng.random((B, H, T, D)), rng.standard_normal((B, H, T, D))
    h0 = rng.standard_normal((B, H, D))
    o, hT = O.scan_fwd(g, x, h0, complement)
    # every channel a head of its own: S_t = exp(g) S + 1 * v, o = 1 * S
    as_heads = lambda t: t.transpose(0, 1, 3, 2).reshape(B, H * D, T, 1)  # noqa: E731
    one = np.ones((B, H * D, T, 1))
    v = as_heads((1 - np.exp(g)) * x if complement else x)
    ro, rS = O.gla_fwd(one, one, v, as_heads(g), h0.reshape(B, H * D, 1, 1))
    np.testing.assert_allclose(as_heads(o), ro, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(hT.reshape(B, H * D, 1, 1), rS, rtol=1e-12, atol=1e-12)


def test_scan_reset_forgets(rng):
    g, x = -rng.random((1, 1, 8, 3)), rng.standard_normal((1, 1, 8, 3))
    g[:, :, 5] = -np.inf
    o, _ = O.scan_fwd(g, x)
    tail, _ = O.scan_fwd(g[:, :, 5:], x[:, :, 5:])
    np.testing.assert_allclose(o[:, :, 5:], tail)
    dg, _, _ = O.scan_bwd(g, x, np.ones_like(x))
    assert np.all(dg[:, :, 5] == 0)


@pytest.mark.parametrize("complement", [False, True])
def test_scan_backward_equals_differences(rng, complement):
    B, H, T, D = 1, 2, 5, 3
    g, x = -rng.random((B, H, T, D)), rng.standard_normal((B, H, T, D))
    h0, do, dhT = rng.standard_normal((B, H, D)), rng.standard_normal((B, H, T, D)), rng.standard_normal((B, H, D))
    f = lambda: O.scan_fwd(g, x, h0, complement)  # noqa: E731
    for got, leaf in zip(O.scan_bwd(g, x, do, h0, dhT, complement), (g, x, h0)):
        np.testing.assert_allclose(got, _diff(f, leaf, (do, dhT)), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("kind", ["group", "rms"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("rows,layout", [(1, "bhtd"), (2, "bthd")])
def test_norm_backward_equals_differences(rng, kind, act, gate, rows, layout):
    B, H, T, D = 2, 2, 3, 4
    x = rng.standard_normal((B, H, T, D) if layout == "bhtd" else (B, T, H, D))
    z = rng.standard_normal((B, T, H, D)) if gate else None
    w, b, dy = rng.standard_normal((rows, D)), rng.standard_normal((rows, D)), rng.standard_normal((B, T, H, D))
    how = dict(kind=kind, act=act, eps=1e-3, layout=layout)
    f = lambda: (O.group_norm_fwd(x, z, w, b, **how),)  # noqa: E731
    for got, leaf in zip(O.group_norm_bwd(x, dy, z, w, b, **how), (x, z, w, b)):
        if leaf is not None:
            np.testing.assert_allclose(got, _diff(f, leaf, (dy,)), rtol=1e-5, atol=1e-7)


def test_norm_equals_torch(rng):
    x = rng.standard_normal((2, 3, 4, 16))
    y = O.group_norm_fwd(x, kind="group", act="none", eps=1e-5)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (16,), eps=1e-5).numpy().transpose(0, 2, 1, 3)
    np.testing.assert_allclose(y, ref, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_complex_multiplication(rng, interleaved):
    x = rng.standard_normal((2, 3, 5, 10))
    freq, pos = rng.random(3), rng.integers(0, 1000, (2, 5))
    y = O.rotary(x, freq, pos, interleaved, scale=1.5)
    pair = (lambda t: t[..., 0:6:2] + 1j * t[..., 1:6:2]) if interleaved else (lambda t: t[..., :3] + 1j * t[..., 3:6])
    np.testing.assert_allclose(pair(y), 1.5 * pair(x) * np.exp(1j * pos[:, None, :, None] * freq), rtol=1e-12)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    back = O.rotary(y, freq, pos, interleaved, scale=1 / 1.5, inverse=True)
    np.testing.assert_allclose(back, x, rtol=1e-12, atol=1e-12)
    dy = rng.standard_normal(x.shape)  # the backward is the transpose
    np.testing.assert_allclose((y * dy).sum(), (x * O.rotary(dy, freq, pos, interleaved, 1.5, True)).sum(), rtol=1e-12)


def test_rotary_frequencies():
    freq, scale = gla.rotary_frequencies(8, device="cpu")
    assert freq.dtype == torch.float64 and scale == 1.0
    np.testing.assert_allclose(freq.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    lin, _ = gla.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(lin.numpy(), freq.numpy() / 4, rtol=1e-14)
    ntk, _ = gla.rotary_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0
    np.testing.assert_allclose(ntk[-1].item(), freq[-1].item() / 4, rtol=1e-12)  # the slowest pair is interpolated
    f, s = gla.rotary_frequencies(64, scaling="yarn", factor=8.0, trained=4096, device="cpu")
    plain, _ = gla.rotary_frequencies(64, device="cpu")
    turns = 4096 * plain.numpy() / (2 * np.pi)
    ratio = f.numpy() / plain.numpy()
    assert np.all(ratio[turns > 64] == 1.0) and np.allclose(ratio[turns < 0.5], 1 / 8)
    assert np.all(np.diff(ratio) <= 1e-12)
    assert s == pytest.approx(0.1 * np.log(8.0) + 1)
    for bad in (dict(R=7), dict(R=0), dict(R=8, base=1.0), dict(R=8, factor=0.5), dict(R=8, scaling="yarn"),
                dict(R=2, scaling="ntk"), dict(R=8, scaling="cubic")):
        with pytest.raises(gla.GLAError):
            gla.rotary_frequencies(device="cpu", **bad)
