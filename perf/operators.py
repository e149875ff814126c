"""Measured cases of the operators that stand around the chunkwise recurrences: the elementwise gated
scan, the per-head group norm with an output gate, and rotary positions.

``run`` computes them in plain torch (``own`` false) or through the library's binding (``own`` true).

    scan    h_t = a_t h_{t-1} + b_t, a = exp(g), b = x or (1 - a) x          g, x [B, H, T, D]
    norm    y = (normalise(x) w + c) act(z)                                  x [B, H, T, D] -> y [B, T, H, D]
    rotary  rotation of the pairs of the first R of D channels by pos * freq q, k -> q', k'
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # One decoded token of 32 requests through a layer 2048 channels wide (the 1.3B layer's 4 x 512).
        {"name": "scan step", "op": "scan_step", "dtype": "bf16", "B": 32, "H": 1, "T": 1, "D": 2048, "complement": True},
        # The prompt of one long request, with few channels to spread over the machine (4 heads of 256).
        {"name": "scan long prompt", "op": "scan_fwd", "dtype": "bf16", "B": 1, "H": 4, "T": 32768, "D": 256, "complement": False},
        # A training batch of the 1.3B layer, channels last.
        {"name": "scan train wide", "op": "scan_train", "dtype": "bf16", "B": 8, "H": 1, "T": 2048, "D": 2048, "complement": True},
        # 32-bit training at a length and a width that no tile divides.
        {"name": "scan train ragged f32", "op": "scan_train", "dtype": "f32", "B": 3, "H": 2, "T": 1531, "D": 333, "complement": False},
        # One decoded token of 8 requests behind the 340M layer.
        {"name": "norm step", "op": "norm_fwd", "dtype": "bf16", "B": 8, "H": 4, "T": 1, "D": 256, "kind": "rms", "act": "silu",
         "gate": True, "shared": True, "layout": "bhtd"},
        # A training batch of the 1.3B layer: four heads of 512, a norm weight for each channel.
        {"name": "norm train", "op": "norm_train", "dtype": "bf16", "B": 8, "H": 4, "T": 2048, "D": 512, "kind": "group", "act": "silu",
         "gate": True, "shared": False, "layout": "bhtd"},
        # 32-bit training, one weight shared by the heads, a head width that 16-byte vectors do not divide.
        {"name": "norm train odd f32", "op": "norm_train", "dtype": "f32", "B": 2, "H": 3, "T": 1021, "D": 130, "kind": "rms", "act": "sigmoid",
         "gate": True, "shared": True, "layout": "bhtd"},
        # A whole layer width as one group behind the scan of a long prompt, already channels last, no gate.
        {"name": "norm wide prompt", "op": "norm_fwd", "dtype": "bf16", "B": 1, "H": 1, "T": 32768, "D": 1024, "kind": "rms", "act": "none",
         "gate": False, "shared": False, "layout": "bthd"},
        # One token each of 16 requests at far positions.
        {"name": "rotary step", "op": "rotary", "dtype": "bf16", "B": 16, "H": 8, "Hk": 8, "T": 1, "D": 128, "R": 128, "interleaved": False,
         "layout": "bhtd", "far": 1000000, "backward": False},
        # The projections' channels-last q, k of a training batch turned into the operators' head-major layout.
        {"name": "rotary train", "op": "rotary", "dtype": "bf16", "B": 8, "H": 4, "Hk": 4, "T": 2048, "D": 256, "R": 256, "interleaved": False,
         "layout": "bthd", "far": 0, "backward": False},
        # Gradients of a long sequence, half of each head rotated, fewer key heads than query heads.
        {"name": "rotary gradient", "op": "rotary", "dtype": "bf16", "B": 1, "H": 8, "Hk": 2, "T": 32768, "D": 128, "R": 64, "interleaved": True,
         "layout": "bhtd", "far": 0, "backward": True},
        # 32-bit, ragged everywhere.
        {"name": "rotary ragged f32", "op": "rotary", "dtype": "f32", "B": 3, "H": 5, "Hk": 1, "T": 509, "D": 90, "R": 50, "interleaved": False,
         "layout": "bthd", "far": 30000, "backward": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_fwd", "scan_train", "scan_train", "norm_fwd", "norm_train", "norm_train", "rotary", "rotary"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    token = op == "scan_step"
    if op.startswith("scan"):
        c.update(B=_log_int(rng, 1, 64 if token else 16), H=rng.choice([1, 1, 2, 4, 7]), T=1 if token else _log_int(rng, 2, 32768),
                 D=rng.choice([_log_int(rng, 8, 2048), 8 * _log_int(rng, 1, 256), 64 * rng.randint(1, 32)]), complement=rng.random() < 0.5)
    elif op.startswith("norm"):
        c.update(B=_log_int(rng, 1, 16), H=rng.choice([1, 2, 4, 4, 5, 16]), T=_log_int(rng, 1, 32768),
                 D=rng.choice([_log_int(rng, 16, 1024), 8 * _log_int(rng, 2, 128), 64 * rng.randint(1, 8)]), kind=rng.choice(["group", "rms"]),
                 act=rng.choice(["silu", "silu", "sigmoid", "none"]), gate=rng.random() < 0.8, shared=rng.random() < 0.5,
                 layout=rng.choice(["bhtd", "bhtd", "bthd"]))
    else:
        D = rng.choice([64, 128, 256, 2 * _log_int(rng, 8, 128)])
        H = rng.choice([1, 4, 8, 9, 16])
        c.update(B=_log_int(rng, 1, 16), H=H, Hk=rng.choice([H, 1, 2]), T=_log_int(rng, 1, 32768), D=D, R=rng.choice([D, D, D // 2 // 2 * 2]),
                 interleaved=rng.random() < 0.5, layout=rng.choice(["bhtd", "bthd"]), far=rng.choice([0, 0, 50000, 1000000]),
                 backward=rng.random() < 0.5)
    most = {"scan_step": 2e7}.get(op, 5.2e8)
    while work(c)["bytes"] > most:
        if c["B"] > 1 and c["B"] >= c["T"] // 256:
            c["B"] = max(1, c["B"] * 2 // 3)
        else:
            c["T"] = c["T"] * 2 // 3 + 1
    return c


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rotary":
        heads, tokens = c["H"] + c["Hk"], c["B"] * c["T"]
        return {"bytes": 2 * size * tokens * heads * c["D"] + 8 * c["T"] + 4 * c["R"], "flops": tokens * heads * c["R"] * 3}
    n = c["B"] * c["H"] * c["T"] * c["D"]
    if c["op"].startswith("scan"):
        rows = 4 * c["B"] * c["H"] * c["D"]  # one 32-bit state
        if c["op"] == "scan_train":
            return {"bytes": 8 * size * n + 4 * rows, "flops": 16 * n}  # forward g, x -> o; backward g, x, do -> dg, dx; h0, hT, dhT, dh0
        return {"bytes": 3 * size * n + 2 * rows, "flops": 5 * n}
    weights = 8 * c["D"] * (1 if c["shared"] else c["H"])
    gate = 1 if c["gate"] else 0
    if c["op"] == "norm_train":
        return {"bytes": (5 + 3 * gate) * size * n + 3 * weights, "flops": 40 * n}
    return {"bytes": (2 + gate) * size * n + weights, "flops": 12 * n}


def _frequencies(R):
    """Radians a position for each pair, in 64 bits: 10000^(-2 i / R)."""
    return 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dtype):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    s = {"case": c}
    if c["op"] == "rotary":
        def per_token(H, layout):
            return normal(c["B"], c["T"], H, c["D"]) if layout == "bthd" else normal(c["B"], H, c["T"], c["D"])

        # gradients come in the layout of the rotated tensors, which is head-major
        layout = "bhtd" if c["backward"] else c["layout"]
        s["q"], s["k"] = per_token(c["H"], layout), per_token(c["Hk"], layout)
        s["freq"] = _frequencies(c["R"])
        start = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=gen, device="cuda")
        s["pos"] = start + torch.arange(c["T"], device="cuda")
        return s
    B, H, T, D = c["B"], c["H"], c["T"], c["D"]
    if c["op"].startswith("scan"):
        shape = (B, H, D) if c["op"] == "scan_step" else (B, H, T, D)
        logits = torch.randn(shape, generator=gen, device="cuda")
        s["g"] = (torch.nn.functional.logsigmoid(logits) / 16).to(dtype)
        s["x"] = normal(*shape)
        s["h0"] = normal(B, H, D, dtype=torch.float32)
        if c["op"] == "scan_train":
            s["do"] = normal(*shape)
            s["dhT"] = normal(B, H, D, dtype=torch.float32)
        return s
    s["x"] = normal(B, H, T, D) if c["layout"] == "bhtd" else normal(B, T, H, D)
    s["z"] = normal(B, T, H, D) if c["gate"] else None
    rows = 1 if c["shared"] else H
    s["w"] = 1 + 0.1 * normal(rows, D, dtype=torch.float32)
    s["c"] = 0.1 * normal(rows, D, dtype=torch.float32)
    if c["op"] == "norm_train":
        s["dy"] = normal(B, T, H, D)
    return s


# ---------------------------------------------------------------------------- plain forms
def _plain_scan(a, b, first):
    """h_t = a_t h_{t-1} + b_t along the third axis from the state `first`, by doubling the reach of each token's sum."""
    h = b.clone()
    h[:, :, 0] += a[:, :, 0] * first
    a = a.clone()
    reach, T = 1, a.shape[2]
    while reach < T:
        h[:, :, reach:] = h[:, :, reach:] + a[:, :, reach:] * h[:, :, :-reach]
        a[:, :, reach:] = a[:, :, reach:] * a[:, :, :-reach]
        reach *= 2
    return h


def _plain_scan_run(s, c):
    g, x = s["g"].float(), s["x"].float()
    a = g.exp()
    share = -torch.expm1(g) if c["complement"] else None
    b = x * share if c["complement"] else x
    if c["op"] == "scan_step":
        s["h0"].copy_(a * s["h0"] + b)
        return {"o": s["h0"].to(s["x"].dtype), "h": s["h0"]}
    h = _plain_scan(a, b, s["h0"])
    out = {"o": h.to(s["x"].dtype), "hT": h[:, :, -1].contiguous()}
    if c["op"] == "scan_train":
        do = s["do"].float()
        after = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], 2)  # a_{t+1}; the last token takes dhT as it is
        d = _plain_scan(after.flip(2), do.flip(2), s["dhT"]).flip(2)
        before = torch.cat([s["h0"].unsqueeze(2), h[:, :, :-1]], 2)
        dg = a * (before - x) * d if c["complement"] else a * before * d
        dx = share * d if c["complement"] else d
        out.update(dg=dg.to(s["x"].dtype), dx=dx.to(s["x"].dtype), dh0=a[:, :, 0] * d[:, :, 0])
    return out


def _plain_act(v, act):
    """act(v) and its derivative."""
    if act == "none":
        return v, torch.ones_like(v)
    e = 1 / (1 + torch.exp(-v))
    if act == "sigmoid":
        return e, e * (1 - e)
    return v * e, e * (1 + v * (1 - e))


def _plain_norm_run(s, c):
    x = s["x"].float()
    if c["layout"] == "bhtd":
        x = x.transpose(1, 2)
    mean = x.mean(-1, keepdim=True) if c["kind"] == "group" else 0.0
    n = x - mean
    rstd = 1 / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS)
    n = n * rstd
    u = n * s["w"] + s["c"]
    if c["gate"]:
        z = s["z"].float()
        f, slope = _plain_act(z, c["act"])
        y = u * f
    else:
        y, slope = _plain_act(u, c["act"])
    out = {"y": y.to(s["x"].dtype)}
    if c["op"] == "norm_train":
        dy = s["dy"].float()
        du = dy * f if c["gate"] else dy * slope
        if c["gate"]:
            out["dz"] = (dy * u * slope).to(s["x"].dtype)
        over = (0, 1, 2) if c["shared"] else (0, 1)
        out["dw"] = (du * n).sum(over).reshape(s["w"].shape)
        out["dc"] = du.sum(over).reshape(s["w"].shape)
        dn = du * s["w"]
        dx = dn - n * (dn * n).mean(-1, keepdim=True)
        if c["kind"] == "group":
            dx = dx - dn.mean(-1, keepdim=True)
        dx = (dx * rstd).to(s["x"].dtype)
        out["dx"] = dx.transpose(1, 2).contiguous() if c["layout"] == "bhtd" else dx
    return out


def _plain_rotate(x, angle, c):
    """x [B, T, H, D] with its first R channels rotated by angle [B, T, 1, R / 2]."""
    R = c["R"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    p = x[..., 0:R:2] if c["interleaved"] else x[..., : R // 2]
    q = x[..., 1:R:2] if c["interleaved"] else x[..., R // 2 : R]
    first, second = p * cos - q * sin, q * cos + p * sin
    turned = torch.stack([first, second], -1).flatten(-2) if c["interleaved"] else torch.cat([first, second], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rotary_run(s, c):
    angle = (s["pos"].double().unsqueeze(-1) * s["freq"]).unsqueeze(2)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if c["backward"]:  # head-major gradients back to the layout of the inputs
            y = _plain_rotate(x.transpose(1, 2), -angle, c)
            y = y if c["layout"] == "bthd" else y.transpose(1, 2)
        else:
            y = _plain_rotate(x if c["layout"] == "bthd" else x.transpose(1, 2), angle, c).transpose(1, 2)
        out[name] = y.to(s[name].dtype).contiguous()
    return out


# ---------------------------------------------------------------------------- the library's calls
def _own_run(s, c):
    from chunkwise_linear_rnn_02_b200 import binding as gla

    op = c["op"]
    if op == "scan_step":
        return {"o": gla.scan_step(s["g"], s["x"], s["h0"], complement=c["complement"]), "h": s["h0"]}
    if op == "scan_fwd":
        o, hT, _ = gla.scan_fwd(s["g"], s["x"], h0=s["h0"], complement=c["complement"])
        return {"o": o, "hT": hT}
    if op == "scan_train":
        o, hT, hc = gla.scan_fwd(s["g"], s["x"], h0=s["h0"], complement=c["complement"], save_states=True)
        dg, dx, dh0 = gla.scan_bwd(s["g"], s["x"], s["do"], h0=s["h0"], dhT=s["dhT"], hc=hc, complement=c["complement"])
        return {"o": o, "hT": hT, "dg": dg, "dx": dx, "dh0": dh0}
    if op.startswith("norm"):
        how = {"kind": c["kind"], "act": c["act"], "eps": EPS, "layout": c["layout"]}
        out = {"y": gla.group_norm_fwd(s["x"], z=s["z"], w=s["w"], b=s["c"], **how)}
        if op == "norm_train":
            out["dx"], dz, out["dw"], out["dc"] = gla.group_norm_bwd(s["x"], s["dy"], z=s["z"], w=s["w"], b=s["c"], **how)
            if dz is not None:
                out["dz"] = dz
        return out
    turn = gla.rotary_bwd if c["backward"] else gla.rotary
    q, k = turn(s["q"], s["k"], s["freq"], pos=s["pos"], interleaved=c["interleaved"], layout=c["layout"])
    return {"q": q, "k": k}


def run(state):
    c = state["case"]
    if own:
        return _own_run(state, c)
    if c["op"].startswith("scan"):
        return _plain_scan_run(state, c)
    return _plain_norm_run(state, c) if c["op"].startswith("norm") else _plain_rotary_run(state, c)


# ---------------------------------------------------------------------------- 64 bits, from the definitions
def _exact_scan(s, c):
    g, x, h = s["g"].double(), s["x"].double(), s["h0"].double()
    if c["op"] == "scan_step":
        a = torch.exp(g)
        h = a * h + (x - a * x if c["complement"] else x)
        return {"o": h, "h": h}
    T = c["T"]
    states = torch.empty(T + 1, *h.shape, dtype=torch.float64, device=h.device)
    states[0] = h
    a = torch.exp(g).permute(2, 0, 1, 3).contiguous()
    x = x.permute(2, 0, 1, 3).contiguous()
    b = x - a * x if c["complement"] else x
    for t in range(T):
        torch.addcmul(b[t], a[t], states[t], out=states[t + 1])
    out = {"o": states[1:].permute(1, 2, 0, 3), "hT": states[T]}
    if c["op"] == "scan_train":
        do = s["do"].double().permute(2, 0, 1, 3).contiguous()
        d = torch.empty_like(do)
        back = s["dhT"].double()
        for t in range(T - 1, -1, -1):
            torch.add(do[t], back, out=d[t])
            back = a[t] * d[t]
        # h_t = h_{t-1} a_t + b_t: d h_t / d g_t = a_t (h_{t-1} - [complement] x_t)
        da = d * (states[:-1] - x if c["complement"] else states[:-1])
        dx = d - a * d if c["complement"] else d
        out.update(dg=(da * a).permute(1, 2, 0, 3), dx=dx.permute(1, 2, 0, 3), dh0=back)
    return out


def _exact_norm(s, c):
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "z", "w", "c") if s[k] is not None}
    x = leaf["x"] if c["layout"] == "bthd" else leaf["x"].permute(0, 2, 1, 3)
    if c["kind"] == "group":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        u = (x - mean) * torch.rsqrt(var + EPS)
    else:
        u = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    u = u * leaf["w"] + leaf["c"]
    v = leaf["z"] if c["gate"] else u
    f = {"none": v, "sigmoid": torch.sigmoid(v), "silu": v * torch.sigmoid(v)}[c["act"]]
    y = u * f if c["gate"] else f
    out = {"y": y.detach()}
    if c["op"] == "norm_train":
        names = sorted(leaf)
        grads = dict(zip(names, torch.autograd.grad(y, [leaf[n] for n in names], s["dy"].double())))
        out.update({"d" + n: grads[n] for n in names})
    return out


def _exact_rotary(s, c):
    B, T, R = c["B"], c["T"], c["R"]
    phase = torch.polar(torch.ones(B, T, R // 2, dtype=torch.float64, device="cuda"), s["pos"].double()[..., None] * s["freq"])
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        head_major = c["backward"] or c["layout"] == "bhtd"
        turn = (phase.conj() if c["backward"] else phase)
        turn = turn[:, None] if head_major else turn[:, :, None]
        pairs = x[..., :R].unflatten(-1, (R // 2, 2) if c["interleaved"] else (2, R // 2))
        axis = -1 if c["interleaved"] else -2
        z = torch.complex(pairs.select(axis, 0), pairs.select(axis, 1)) * turn
        y = torch.cat([torch.stack([z.real, z.imag], axis).flatten(-2), x[..., R:]], -1)
        swap = (c["layout"] == "bthd") if c["backward"] else not head_major
        out[name] = y.transpose(1, 2) if swap else y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("scan"):
        return _exact_scan(s, case)
    return _exact_norm(s, case) if case["op"].startswith("norm") else _exact_rotary(s, case)
