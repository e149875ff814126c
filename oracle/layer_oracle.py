"""Plain fp64 CPU oracle for the operators around the recurrences: the elementwise gated scan, the
group norm with an output gate, and rotary positions.

TEST INFRASTRUCTURE ONLY, like the other oracles: numpy, written as the definitions.  The reverse modes
are hand-derived; the tests check them against central differences.

* scan: h_t = a_t h_{t-1} + b_t with a = exp(g) and b = x, or b = (1 - a) x.
* group norm: every head of a token is one group of D values; n = (x - mean) / sqrt(var + eps) or
  x / sqrt(mean x^2 + eps); u = n w + b; y = u act(z), or act(u) without z.  y, z are [B,T,H,D].
* rotary: pairs of the first R channels turned by p * freq_i.
"""
from __future__ import annotations

import numpy as np

__all__ = ["scan_fwd", "scan_bwd", "group_norm_fwd", "group_norm_bwd", "rotary"]


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def scan_fwd(g, x, h0=None, complement=False):
    """[B,H,T,D] -> (o [B,H,T,D], hT [B,H,D])."""
    g, x = _f(g), _f(x)
    h = np.zeros(g.shape[:2] + g.shape[3:]) if h0 is None else _f(h0).copy()
    o = np.empty_like(x)
    for t in range(g.shape[2]):
        a = np.exp(g[:, :, t])
        b = -np.expm1(g[:, :, t]) * x[:, :, t] if complement else x[:, :, t]
        h = a * h + b
        o[:, :, t] = h
    return o, h


def scan_bwd(g, x, do, h0=None, dhT=None, complement=False):
    """Gradients of sum(do * o) + sum(dhT * hT): (dg, dx, dh0)."""
    g, x, do = _f(g), _f(x), _f(do)
    o, _ = scan_fwd(g, x, h0, complement)
    first = np.zeros(g.shape[:2] + g.shape[3:]) if h0 is None else _f(h0)
    back = np.zeros_like(first) if dhT is None else _f(dhT).copy()
    dg, dx = np.empty_like(g), np.empty_like(x)
    for t in range(g.shape[2] - 1, -1, -1):
        a = np.exp(g[:, :, t])
        before = first if t == 0 else o[:, :, t - 1]
        d = do[:, :, t] + back
        back = a * d
        dx[:, :, t] = -np.expm1(g[:, :, t]) * d if complement else d
        dg[:, :, t] = back * (before - x[:, :, t] if complement else before)
    return dg, dx, back


def _act(v, act):
    if act == "none":
        return v, np.ones_like(v)
    s = 1.0 / (1.0 + np.exp(-v))
    if act == "sigmoid":
        return s, s * (1 - s)
    return v * s, s * (1 + v * (1 - s))


def _norm(x, w, b, kind, eps, layout):
    x = _f(x)
    if layout == "bhtd":
        x = x.transpose(0, 2, 1, 3)
    c = x - x.mean(-1, keepdims=True) if kind == "group" else x
    rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = c * rstd
    w = np.ones((1, x.shape[-1])) if w is None else _f(w)
    return n, rstd, w, n * w + (0.0 if b is None else _f(b))


def group_norm_fwd(x, z=None, w=None, b=None, kind="group", act="silu", eps=1e-5, layout="bhtd"):
    _, _, _, u = _norm(x, w, b, kind, eps, layout)
    return _act(u, act)[0] if z is None else u * _act(_f(z), act)[0]


def group_norm_bwd(x, dy, z=None, w=None, b=None, kind="group", act="silu", eps=1e-5, layout="bhtd"):
    """(dx in x's layout, dz or None, dw, db), the last two summed to the rows of w and b ([1,D] when None)."""
    n, rstd, ww, u = _norm(x, w, b, kind, eps, layout)
    dy = _f(dy)
    if z is None:
        dz, du = None, dy * _act(u, act)[1]
    else:
        f, slope = _act(_f(z), act)
        dz, du = dy * u * slope, dy * f
    over = (0, 1) if ww.shape[0] > 1 else (0, 1, 2)
    dw, db = (du * n).sum(over).reshape(ww.shape), du.sum(over).reshape(ww.shape)
    dn = du * ww
    dx = dn - n * (dn * n).mean(-1, keepdims=True)
    if kind == "group":
        dx = dx - dn.mean(-1, keepdims=True)
    dx = dx * rstd
    return (dx.transpose(0, 2, 1, 3) if layout == "bhtd" else dx), dz, dw, db


def rotary(x, freq, pos, interleaved=False, scale=1.0, inverse=False):
    """x [B,H,T,D], pos [B,T]; pairs (u, v) -> scale (u cos - v sin, v cos + u sin)."""
    x, freq = _f(x), _f(freq)
    R = 2 * len(freq)
    A = np.asarray(pos, dtype=np.float64)[:, None, :, None] * freq
    c, s = scale * np.cos(A), scale * np.sin(-A if inverse else A)
    u, v = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2 : R])
    y = x.copy()
    if interleaved:
        y[..., 0:R:2], y[..., 1:R:2] = u * c - v * s, v * c + u * s
    else:
        y[..., : R // 2], y[..., R // 2 : R] = u * c - v * s, v * c + u * s
    return y
