"""The operators as a layer uses them, one after another on the GPU, forward and backward, against the fp64
oracle's composition: rotary q, k -> chunkwise GLA -> group norm with an output gate, and the elementwise scan
-> the same norm.  Each stage is held to the library's bf16 / fp32 parity bound on its own inputs (the oracle gets
what the stage before it returned), so the bound does not grow along the run."""
import pytest
import torch

import oracle as O
from chunkwise_linear_rnn_02_b200 import binding as gla
from chunkwise_linear_rnn_02_b200.inputs import make_gla_inputs
from helpers import assert_close, f64, tol_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_retention_layer(dtype):
    B, H, T, dk, dv = 2, 2, 200, 64, 128
    tol = tol_for(dtype)
    c = {k: v.cuda() for k, v in make_gla_inputs(B, H, T, dk, dv, dtype, seed=1).items()}
    gen = torch.Generator().manual_seed(2)
    z, dy = (torch.randn(B, T, H, dv, generator=gen).to(dtype).cuda() for _ in range(2))
    w, b = (1 + torch.randn(H, dv, generator=gen) / 8).cuda(), (torch.randn(H, dv, generator=gen) / 8).cuda()
    freq, scale = gla.rotary_frequencies(dk)
    how = dict(kind="group", act="silu", layout="bhtd")
    q, k = gla.rotary(c["q"], c["k"], freq, scale=scale)
    o, _ = gla.chunk_fwd(q, k, c["v"], c["g"])
    y = gla.group_norm_fwd(o, z, w, b, **how)
    do, dz, dw, db = gla.group_norm_bwd(o, dy, z, w, b, **how)
    dq, dkk, dvv, dg, _ = gla.chunk_bwd(q, k, c["v"], c["g"], do)
    dq0, dk0 = gla.rotary_bwd(dq, dkk, freq, scale=scale)
    pos = [list(range(T))] * B
    assert_close("q", q, O.rotary(f64(c["q"]), f64(freq), pos), tol)
    assert_close("k", k, O.rotary(f64(c["k"]), f64(freq), pos), tol)
    assert_close("o", o, O.gla_fwd(f64(q), f64(k), f64(c["v"]), f64(c["g"]))[0], tol)
    assert_close("y", y, O.group_norm_fwd(f64(o), f64(z), f64(w), f64(b), **how), tol)
    for n, got, ref in zip(("do", "dz", "dw", "db"), (do, dz, dw, db),
                           O.group_norm_bwd(f64(o), f64(dy), f64(z), f64(w), f64(b), **how)):
        assert_close(n, got, ref, tol)
    for n, got, ref in zip(("dq", "dk", "dv", "dg"), (dq, dkk, dvv, dg),
                           O.gla_bwd(f64(q), f64(k), f64(c["v"]), f64(c["g"]), None, f64(do))):
        assert_close(n, got, ref, tol)
    assert_close("dq0", dq0, O.rotary(f64(dq), f64(freq), pos, inverse=True), tol)
    assert_close("dk0", dk0, O.rotary(f64(dkk), f64(freq), pos, inverse=True), tol)
    assert gla.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scan_layer_prompt_then_tokens(dtype):
    """Gate logits -> gate -> scan -> norm over a prompt, then token by token from its final state: the tokens
    equal what one longer prompt gives."""
    B, T, new, C, G = 2, 150, 4, 96, 3
    tol = tol_for(dtype)
    gen = torch.Generator().manual_seed(3)
    logits, x = (torch.randn(B, 1, T + new, C, generator=gen).to(dtype).cuda() for _ in range(2))
    z = torch.randn(B, T + new, G, C // G, generator=gen).to(dtype).cuda()
    w = (1 + torch.randn(1, C // G, generator=gen) / 8).cuda()
    g = gla.gate_logsigmoid(logits, 8.0)
    how = dict(kind="rms", act="silu", layout="bthd")
    o, _, _ = gla.scan_fwd(g, x, complement=True)
    whole = gla.group_norm_fwd(o.view(B, T + new, G, C // G), z, w, **how)
    cut = lambda t: t[:, :, :T].contiguous()  # noqa: E731
    first, S, hc = gla.scan_fwd(cut(g), cut(x), complement=True, save_states=True)
    assert_close("o", first, O.scan_fwd(f64(cut(g)), f64(cut(x)), None, True)[0], tol)
    for t in range(T, T + new):
        ot = gla.scan_step(g[:, :, t].contiguous(), x[:, :, t].contiguous(), S, complement=True)
        yt = gla.group_norm_fwd(ot.view(B, 1, G, C // G), z[:, t:t + 1].contiguous(), w, **how)
        assert_close("y", yt[:, 0], f64(whole[:, t]), tol)
    # and the gradients of the prompt, back to the gate logits
    dy = torch.randn(B, T, G, C // G, generator=gen).to(dtype).cuda()
    do, _, dw, _ = gla.group_norm_bwd(first.view(B, T, G, C // G), dy, z[:, :T].contiguous(), w, **how)
    do = do.view(B, 1, T, C)
    dg, dx, _ = gla.scan_bwd(cut(g), cut(x), do, hc=hc, complement=True)
    dlogits = gla.gate_logsigmoid_bwd(cut(logits), dg, 8.0)
    rg, rx, _ = O.scan_bwd(f64(cut(g)), f64(cut(x)), f64(do), None, None, True)
    assert_close("dg", dg, rg, tol)
    assert_close("dx", dx, rx, tol)
    assert_close("dlogits", dlogits, O.gate_logsigmoid_bwd(f64(cut(logits)), f64(dg), 8.0), tol)
    rdo, _, rdw, _ = O.group_norm_bwd(f64(first).reshape(B, T, G, C // G), f64(dy), f64(z[:, :T]), f64(w), None, **how)
    assert_close("do", do, rdo.reshape(B, 1, T, C), tol)
    assert_close("dw", dw, rdw, tol)


def test_two_threads_at_once():
    """The scan's and the norm's backward from two host threads on streams of their own: the bits of each alone."""
    import threading

    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    g, x, do = -r(1, 2, 5000, 64).abs() / 16, r(1, 2, 5000, 64), r(1, 2, 5000, 64)
    nx, nz, ndy = r(4, 4, 700, 128), r(4, 700, 4, 128), r(4, 700, 4, 128)
    w, b = torch.randn(4, 128, generator=gen).cuda(), torch.randn(4, 128, generator=gen).cuda()
    jobs = [lambda: gla.scan_bwd(g, x, do, complement=True), lambda: gla.group_norm_bwd(nx, ndy, nz, w, b)]
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                out = jobs[i]()
        s.synchronize()
        got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    for a, o in zip(alone, got):
        assert o is not None and all(torch.equal(p, q) for p, q in zip(a, o))
    assert gla.device_error() == 0
