"""Run the operators on one synthetic case, e.g. to profile a single kernel.

    python -m chunkwise_linear_rnn_02_b200.run_case --op fwd --B 8 --H 4 --T 2048 --dk 128 --dv 256 --iters 3
    python -m chunkwise_linear_rnn_02_b200.run_case --op scan_bwd --B 8 --H 1 --T 2048 --dv 2048

The scan, norm and rotary take their channels a head from --dv.

Inputs follow the seeded recipe of ``inputs.py``.  Prints the mean time per call measured with
CUDA events (not meaningful under a profiler).
"""
from __future__ import annotations

import argparse

import torch

from . import binding as gla
from .inputs import make_gla_inputs, make_gsa_inputs, make_layer_inputs


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", choices=["fwd", "bwd", "fwdbwd", "decode", "gsa_fwd", "gsa_bwd", "scan_fwd", "scan_bwd",
                                     "scan_step", "norm_fwd", "norm_bwd", "rotary"], default="fwdbwd")
    ap.add_argument("--complement", action="store_true", help="scan: h = a h + (1 - a) x")
    ap.add_argument("--B", type=int, default=8)
    ap.add_argument("--H", type=int, default=4)
    ap.add_argument("--T", type=int, default=2048)
    ap.add_argument("--dk", type=int, default=128)
    ap.add_argument("--dv", type=int, default=256)
    ap.add_argument("--m", type=int, default=64)
    ap.add_argument("--chunk", type=int, default=64)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    ap.add_argument("--iters", type=int, default=3)
    a = ap.parse_args(argv)
    dt = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    layer = a.op.startswith(("scan", "norm", "rotary"))
    if layer:
        d = {k: v.cuda() for k, v in make_layer_inputs(a.B, a.H, a.T, a.dv, dt).items()}
        freq, scale = gla.rotary_frequencies(a.dv - a.dv % 2)
        hc = gla.scan_fwd(d["g"], d["x"], complement=a.complement, save_states=True)[2] if a.op == "scan_bwd" else None
    elif a.op.startswith("gsa"):
        d = {k: v.cuda() for k, v in make_gsa_inputs(a.B, a.H, a.T, a.dk, a.dv, a.m, dt).items()}
    else:
        d = {k: v.cuda() for k, v in make_gla_inputs(a.B, a.H, a.T, a.dk, a.dv, dt).items()}

    def call():
        if a.op in ("fwd", "fwdbwd"):
            gla.chunk_fwd(d["q"], d["k"], d["v"], d["g"], chunk=a.chunk)
        if a.op in ("bwd", "fwdbwd"):
            gla.chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], chunk=a.chunk)
        if a.op == "decode":
            S = torch.zeros(a.B, a.H, a.dk, a.dv, device="cuda")
            gla.recurrent_step(d["q"][:, :, 0].contiguous(), d["k"][:, :, 0].contiguous(),
                               d["v"][:, :, 0].contiguous(), d["g"][:, :, 0].contiguous(), S)
        if a.op == "scan_fwd":
            gla.scan_fwd(d["g"], d["x"], complement=a.complement, save_states=True)
        if a.op == "scan_bwd":
            gla.scan_bwd(d["g"], d["x"], d["do"], hc=hc, complement=a.complement)
        if a.op == "scan_step":
            S = torch.zeros(a.B, a.H, a.dv, device="cuda")
            gla.scan_step(d["g"][:, :, 0].contiguous(), d["x"][:, :, 0].contiguous(), S, complement=a.complement)
        if a.op == "norm_fwd":
            gla.group_norm_fwd(d["x"], d["z"], d["w"], d["b"])
        if a.op == "norm_bwd":
            gla.group_norm_bwd(d["x"], d["dy"], d["z"], d["w"], d["b"])
        if a.op == "rotary":
            gla.rotary(d["x"], d["do"], freq, scale=scale)
        if a.op == "gsa_fwd":
            gla.gsa_fwd(d["q"], d["k"], d["v"], d["phi"], d["g"], chunk=a.chunk)
        if a.op == "gsa_bwd":
            gla.gsa_bwd(d["q"], d["k"], d["v"], d["phi"], d["g"], d["do"], chunk=a.chunk)

    call()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(a.iters):
        call()
    e1.record()
    torch.cuda.synchronize()
    print(f"{a.op} B={a.B} H={a.H} T={a.T} dk={a.dk} dv={a.dv}: {e0.elapsed_time(e1) / a.iters:.4f} ms/call "
          f"(device error latch {gla.device_error()})")


if __name__ == "__main__":
    main()
