"""GPU parity of the elementwise scan (forward, backward, single token) against the fp64 oracle.

Tolerances are bounds, not guesses.  A gate's exponential is within 2^-22 relative of the true one
(the approximate base-2 exponential, or five terms of a series), plus the rounding of its argument,
|g| log2(e) 2^-24; the tests keep finite g above -4, so a step's factor is off by less than 2^-21, and the
multiply-add and the joining of runs, blocks and clusters round a few more times per step: EPS = 2^-20 a
step covers both.  A term that has passed through n steps is then off by n EPS of its size, so the error
of a state is at most EPS times the scan of the ages, M_t = a M_{t-1} + N_t with N_t = a N_{t-1} + |b_t|.
The output's own rounding, half a step of its type, comes on top.
"""
import numpy as np
import pytest
import torch

import oracle as O
from chunkwise_linear_rnn_02_b200 import binding as gla
from helpers import f64

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


def make(B, H, T, D, dtype, seed, resets=0, keeps=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = torch.nn.functional.logsigmoid(r(B, H, T, D)) / 4
    # a spread of memories: some channels nearly keep everything, some forget within a token or two
    g = (g * torch.logspace(-2.5, 0.5, D)).clamp(min=-4.0)
    where = torch.rand(B, H, T, D, generator=gen)
    if resets:
        g[where < resets] = -float("inf")
    if keeps:
        g[where > 1 - keeps] = 0.0
    x, do = r(B, H, T, D), r(B, H, T, D)
    h0, dhT = r(B, H, D), r(B, H, D)
    return {"g": g.to(dtype), "x": x.to(dtype), "do": do.to(dtype), "h0": h0, "dhT": dhT}


def bounds(d, complement, with_h0, with_dhT):
    """The oracle's results and the allowed error of each, before the output's rounding."""
    g, x, do = f64(d["g"]), f64(d["x"]), f64(d["do"])
    h0 = f64(d["h0"]) if with_h0 else None
    dhT = f64(d["dhT"]) if with_dhT else None
    o, hT = O.scan_fwd(g, x, h0, complement)
    dg, dx, dh0 = O.scan_bwd(g, x, do, h0, dhT, complement)
    T = g.shape[2]
    b = np.abs(-np.expm1(g) * x if complement else x)

    def ages(g_, b_, first):
        n = np.zeros(first.shape) + np.abs(first)
        m = n.copy()
        N, M = np.empty_like(b_), np.empty_like(b_)
        for t in range(T):
            a = np.exp(g_[:, :, t])
            n = a * n + b_[:, :, t]
            m = a * m + n
            N[:, :, t], M[:, :, t] = n, m
        return N, M

    zero = np.zeros(g.shape[:2] + g.shape[3:])
    _, Mf = ages(g, b, zero if h0 is None else h0)
    flip = lambda t: t[:, :, ::-1]  # noqa: E731
    after = np.concatenate([g[:, :, 1:], np.zeros_like(g[:, :, :1])], 2)
    Nb, Mb = (flip(t) for t in ages(flip(after), np.abs(flip(do)), zero if dhT is None else dhT))
    before = np.concatenate([(zero if h0 is None else h0)[:, :, None], o[:, :, :-1]], 2)
    M_before = np.concatenate([(np.abs(zero if h0 is None else h0))[:, :, None], Mf[:, :, :-1]], 2)
    a, share = np.exp(g), (-np.expm1(g) if complement else np.ones_like(g))
    inner = np.abs(before - x) if complement else np.abs(before)
    size = np.abs(before) + np.abs(x) if complement else np.abs(before)
    tol = {"o": EPS * Mf, "hT": EPS * Mf[:, :, -1], "dx": EPS * share * (Mb + Nb),
           "dg": EPS * a * (Mb * inner + Nb * (M_before + 2 * size)), "dh0": EPS * a[:, :, 0] * (Mb + Nb)[:, :, 0]}
    return {"o": o, "hT": hT, "dg": dg, "dx": dx, "dh0": dh0}, tol


def check(name, got, ref, tol, dtype):
    got = f64(got)
    assert got.shape == ref.shape
    allowed = tol + HALF[dtype] * (np.abs(ref) + tol) + 1e-37  # the last: fp32's flush to zero
    bad = ~(np.abs(got - ref) <= allowed)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, allowed {allowed[bad][0]:.2e}"


def run_all(d, complement, with_h0=True, with_dhT=True, keep=True):
    c = {k: v.cuda() for k, v in d.items()}
    h0 = c["h0"] if with_h0 else None
    dhT = c["dhT"] if with_dhT else None
    o, hT, hc = gla.scan_fwd(c["g"], c["x"], h0=h0, complement=complement, save_states=True)
    dg, dx, dh0 = gla.scan_bwd(c["g"], c["x"], c["do"], h0=h0, dhT=dhT, hc=hc if keep else None, complement=complement)
    return {"o": o, "hT": hT, "dg": dg, "dx": dx, "dh0": dh0}


SHAPES = [
    (1, 1, 1, 1), (2, 3, 1, 64), (1, 2, 2, 7), (2, 1, 63, 24), (1, 3, 64, 128), (3, 1, 65, 100), (2, 2, 127, 8),
    (1, 1, 130, 333), (4, 2, 513, 64), (1, 1, 1025, 16), (2, 1, 700, 1000), (1, 1, 5000, 40), (8, 1, 300, 512),
    (1, 4, 2049, 256), (1, 1, 20000, 9), (40, 4, 70, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,H,T,D", SHAPES)
def test_scan_against_oracle(B, H, T, D, dtype, complement):
    d = make(B, H, T, D, dtype, seed=T * 31 + D, resets=0.002, keeps=0.01)
    ref, tol = bounds(d, complement, True, True)
    got = run_all(d, complement)
    for n in ref:
        check(n, got[n], ref[n], tol[n], F32 if n in ("hT", "dh0") else dtype)
    # without kept states the backward recomputes them: the same arithmetic, the same bits
    again = run_all(d, complement, keep=False)
    for n in ref:
        assert torch.equal(got[n], again[n]), n
    assert gla.device_error() == 0


# Each slab width, with one block and with a cluster, by TMA and copied by the threads, in one step and in several.
VARIANTS = [
    (1, 1, 200, 16), (16, 4, 257, 72), (300, 1, 130, 33), (3, 4, 513, 200), (3, 4, 1025, 65), (40, 4, 257, 24), (40, 2, 257, 65),
    (8, 4, 1025, 24), (16, 1, 1025, 65), (40, 4, 513, 16), (300, 1, 513, 7), (1, 1, 20000, 16), (100, 2, 130, 24), (16, 2, 513, 24),
    (100, 1, 130, 33), (16, 4, 257, 33), (1, 1, 6000, 7), (2, 1, 65, 1001), (4, 1, 1025, 200), (1, 1, 2049, 16),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,H,T,D", VARIANTS)
def test_scan_variants_against_oracle(B, H, T, D, dtype, complement):
    d = make(B, H, T, D, dtype, seed=T * 37 + D, resets=0.001, keeps=0.01)
    ref, tol = bounds(d, complement, True, True)
    got = run_all(d, complement)
    for n in ref:
        check(n, got[n], ref[n], tol[n], F32 if n in ("hT", "dh0") else dtype)
    assert gla.device_error() == 0


# Many rows of few channels: widths and loads that fill the GPU without a cluster, or with a small one.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,H,T,D", [(150, 1, 130, 33), (40, 2, 130, 72), (300, 1, 130, 16), (40, 2, 64, 24),
                                     (40, 1, 130, 24), (100, 1, 513, 16), (300, 1, 130, 64)])
def test_scan_variants_of_many_rows_against_oracle(B, H, T, D, dtype, complement):
    test_scan_variants_against_oracle(B, H, T, D, dtype, complement)


@pytest.mark.parametrize("with_h0,with_dhT", [(False, False), (True, False), (False, True)])
def test_scan_optional_states(with_h0, with_dhT):
    d = make(2, 2, 200, 48, BF16, seed=5)
    ref, tol = bounds(d, False, with_h0, with_dhT)
    got = run_all(d, False, with_h0, with_dhT)
    for n in ref:
        check(n, got[n], ref[n], tol[n], F32 if n in ("hT", "dh0") else BF16)
    c = {k: v.cuda() for k, v in d.items()}
    o, hT, hc = gla.scan_fwd(c["g"], c["x"], output_final_state=False)
    assert hT is None and hc is None
    assert gla.scan_bwd(c["g"], c["x"], c["do"], need_dh0=False)[2] is None


def test_scan_kept_states_are_the_states():
    d = make(2, 1, 300, 72, F32, seed=6)
    o, hT, hc = gla.scan_fwd(d["g"].cuda(), d["x"].cuda(), h0=d["h0"].cuda(), save_states=True)
    assert hc.shape == (2, 1, 5, 72)
    assert torch.equal(hc[:, :, 0].cpu(), d["h0"])
    for n in range(1, 5):  # fp32 outputs are the states, unrounded
        np.testing.assert_allclose(f64(hc[:, :, n]), f64(o[:, :, 64 * n - 1]), rtol=1e-5, atol=1e-6)
    np.testing.assert_allclose(f64(hT), f64(o[:, :, -1]), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("complement", [False, True])
def test_scan_slow_gates_keep_their_digits(complement):
    """Gates around -1e-5 over 8,192 tokens: 1 - a must not come from a rounded a, nor a product of a's drift.
    With a' = a (1 + e), |e| <= 2^-24 (a stored to the nearest fp32), every term is off by up to n 2^-24 after n
    steps whatever the algorithm; the age bound with that much a step, and twice it for the joins, is the tolerance."""
    T = 8192
    d = make(1, 1, T, 32, F32, seed=7)
    d["g"] = -torch.rand(1, 1, T, 32, generator=torch.Generator().manual_seed(1)) * 2e-5
    ref, tol = bounds(d, complement, True, True)
    got = run_all(d, complement)
    for n in ref:  # EPS = 2^-20 a step becomes 2^-22
        check(n, got[n], ref[n], tol[n] / 4, F32)


def test_scan_resets_separate_packed_sequences():
    """-inf gates cut: sequences packed behind one another give what each gives alone, and no gradient crosses."""
    lens = [1, 70, 200, 64, 129]
    T, D = sum(lens), 64
    d = make(1, 1, T, D, F32, seed=8)
    starts = np.cumsum([0] + lens[:-1])
    d["g"][:, :, starts] = -float("inf")
    got = run_all(d, False, with_h0=True, with_dhT=False)
    for s, n in zip(starts, lens):
        part = {k: (v[:, :, s:s + n].contiguous() if v.dim() == 4 else v) for k, v in d.items()}
        ref, tol = bounds(part, False, False, False)
        for name in ("o", "dx", "dg"):
            check(name, got[name][:, :, s:s + n], ref[name], tol[name], F32)
    assert torch.all(got["dg"][:, :, torch.as_tensor(starts)] == 0)
    assert torch.all(got["dh0"] == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_empty_sequence(dtype):
    g = torch.empty(2, 3, 0, 40, dtype=dtype, device="cuda")
    h0 = torch.randn(2, 3, 40, device="cuda")
    o, hT, hc = gla.scan_fwd(g, g, h0=h0, save_states=True)
    assert o.shape == (2, 3, 0, 40) and hc.shape == (2, 3, 0, 40) and torch.equal(hT, h0)
    assert torch.all(gla.scan_fwd(g, g)[1] == 0)
    assert torch.equal(gla.scan_bwd(g, g, g, dhT=h0)[2], h0)
    assert torch.all(gla.scan_bwd(g, g, g, h0=h0, hc=hc)[2] == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,H,D", [(1, 1, 1), (3, 2, 64), (5, 1, 333), (32, 1, 2048)])
def test_scan_step_continues_the_sequence(dtype, complement, B, H, D):
    T = 5
    d = make(B, H, T, D, dtype, seed=D)
    ref, tol = bounds(d, complement, True, False)
    S = d["h0"].cuda()
    for t in range(T):
        o = gla.scan_step(d["g"][:, :, t].contiguous().cuda(), d["x"][:, :, t].contiguous().cuda(), S, complement=complement)
        check("o", o, ref["o"][:, :, t], tol["o"][:, :, t], dtype)
    check("S", S, ref["hT"], tol["hT"], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_scan_of_tensors_off_their_alignment(dtype, shift):
    """Contiguous views that start one, two or four values into their storage give the same bits as aligned copies
    wherever the vector form and the other one share their order of operations, and the oracle's values anyway;
    memory around the outputs is left alone."""
    B, H, T, D = 2, 2, 150, 64
    d = make(B, H, T, D, dtype, seed=9)
    ref, tol = bounds(d, True, True, True)

    def off(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        flat[shift:] = t.reshape(-1).cuda()
        return flat[shift:].view(t.shape)

    c = {k: off(v) for k, v in d.items()}
    o, hT, hc = gla.scan_fwd(c["g"], c["x"], h0=c["h0"], complement=True, save_states=True)
    dg, dx, dh0 = gla.scan_bwd(c["g"], c["x"], c["do"], h0=c["h0"], dhT=c["dhT"], hc=hc, complement=True)
    for n, t in dict(o=o, hT=hT, dg=dg, dx=dx, dh0=dh0).items():
        check(n, t, ref[n], tol[n], F32 if n in ("hT", "dh0") else dtype)


def test_scan_writes_nothing_else():
    """Outputs inside a larger buffer: the words before and behind them stay as they were."""
    import ctypes
    lib = gla.load_library()
    for B, H, T, D in ((2, 1, 70, 40), (1, 2, 333, 9)):
        d = make(B, H, T, D, BF16, seed=10)
        c = {k: v.cuda() for k, v in d.items()}
        n, m, k = B * H * T * D, B * H * D, B * H * (-(-T // 64)) * D
        pad = 64
        buf = {name: torch.full((size + 2 * pad,), 7.0, dtype=dt, device="cuda")
               for name, size, dt in (("o", n, BF16), ("dg", n, BF16), ("dx", n, BF16), ("hT", m, F32), ("dh0", m, F32), ("hc", k, F32))}
        at = {name: t[pad:].data_ptr() for name, t in buf.items()}
        st = torch.cuda.current_stream().cuda_stream
        p = {k_: v.data_ptr() for k_, v in c.items()}
        assert lib.gla_scan_fwd(p["g"], p["x"], p["h0"], at["o"], at["hT"], at["hc"], B, H, T, D, 0, 1, ctypes.c_void_p(st)) == 0
        assert lib.gla_scan_bwd(p["g"], p["x"], None, at["hc"], p["do"], p["dhT"], at["dg"], at["dx"], at["dh0"], B, H, T, D,
                                0, 1, None, 0, ctypes.c_void_p(st)) == 0
        torch.cuda.synchronize()
        for name, t in buf.items():
            assert torch.all(t[:pad] == 7) and torch.all(t[-pad:] == 7), name
            assert torch.isfinite(t).all()


def test_scan_replayed_and_beside_itself():
    """A captured forward and backward replays on new data; two streams at once and repeated calls give equal bits."""
    d = make(1, 2, 3000, 64, BF16, seed=11)
    c = {k: v.cuda() for k, v in d.items()}

    def step():
        o, hT, hc = gla.scan_fwd(c["g"], c["x"], h0=c["h0"], save_states=True)
        return (o, hT) + gla.scan_bwd(c["g"], c["x"], c["do"], h0=c["h0"], dhT=c["dhT"])  # recomputes the states

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    d2 = make(1, 2, 3000, 64, BF16, seed=12)
    for k in c:
        c[k].copy_(d2[k])
    graph.replay()
    torch.cuda.synchronize()
    ref, tol = bounds(d2, False, True, True)
    for n, t in zip(("o", "hT", "dg", "dx", "dh0"), out):
        check(n, t, ref[n], tol[n], F32 if n in ("hT", "dh0") else BF16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(3):
                results.append(step())
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
    assert gla.device_error() == 0


def test_scan_binding_refusals():
    g = torch.zeros(1, 2, 8, 16, device="cuda", dtype=BF16)
    s = torch.zeros(1, 2, 16, device="cuda")
    with pytest.raises(gla.GLAError, match="x must be"):
        gla.scan_fwd(g, g[:, :, :4])
    with pytest.raises(gla.GLAError, match="x must be"):
        gla.scan_fwd(g, g.float())
    with pytest.raises(gla.GLAError, match="contiguous"):
        gla.scan_fwd(g, torch.zeros(1, 2, 16, 8, device="cuda", dtype=BF16).transpose(2, 3))
    with pytest.raises(gla.GLAError, match="h0 must be"):
        gla.scan_fwd(g, g, h0=s.to(BF16))
    with pytest.raises(gla.GLAError, match="hc must be"):
        gla.scan_bwd(g, g, g, hc=torch.zeros(1, 2, 2, 16, device="cuda"))
    with pytest.raises(gla.GLAError, match="unsupported dtype"):
        gla.scan_fwd(g.half(), g.half())
    with pytest.raises(gla.GLAError, match="dimensions"):
        gla.scan_fwd(s, s)
    with pytest.raises(gla.GLAError, match="CUDA"):
        gla.scan_fwd(g, g.cpu())
    with pytest.raises(gla.GLAError, match="S"):
        gla.scan_step(g[:, :, 0].contiguous(), g[:, :, 0].contiguous(), None)
