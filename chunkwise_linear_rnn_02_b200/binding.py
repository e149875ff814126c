"""Thin Python binding of the C ABI in ``include/gla.h`` (ctypes; argument marshalling only).

PyTorch supplies device memory and the current CUDA stream.  Every step of every operator runs
in the CUDA library ``lib/libgla_b200.so``; if that library is missing or the tensors are not
CUDA tensors, the calls raise instead of computing anything elsewhere.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re

import torch

__all__ = [
    "GLAError", "load_library", "library_path", "header_symbols", "status_string", "version",
    "chunk_fwd", "chunk_bwd", "chunk_fwd_logit", "chunk_bwd_logit", "recurrent_step", "gsa_fwd", "gsa_bwd", "gsa_recurrent_step",
    "device_error", "workspace_bytes", "scan_fwd", "scan_bwd", "scan_step", "group_norm_fwd", "group_norm_bwd",
    "rotary", "rotary_bwd", "rotary_frequencies",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_HEADER = os.path.join(os.path.dirname(_HERE), "include", "gla.h")
_LIB = None

DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1}

_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGNATURES = {
    "gla_status_string": (ctypes.c_char_p, [_i]),
    "gla_version": (_i, []),
    "gla_chunk_fwd_workspace": (_sz, [_i] * 7),
    "gla_chunk_fwd": (_i, [_vp] * 7 + [_i] * 7 + [_vp, _sz, _vp]),
    "gla_chunk_bwd_workspace": (_sz, [_i] * 7),
    "gla_chunk_bwd": (_i, [_vp] * 12 + [_i] * 7 + [_vp, _sz, _vp]),
    "gla_chunk_fwd_logit_workspace": (_sz, [_i] * 7),
    "gla_chunk_fwd_logit": (_i, [_vp] * 4 + [ctypes.c_float] + [_vp] * 3 + [_i] * 7 + [_vp, _sz, _vp]),
    "gla_chunk_bwd_logit_workspace": (_sz, [_i] * 7),
    "gla_chunk_bwd_logit": (_i, [_vp] * 4 + [ctypes.c_float] + [_vp] * 8 + [_i] * 7 + [_vp, _sz, _vp]),
    "gla_recurrent_step": (_i, [_vp] * 6 + [_i] * 5 + [_vp]),
    "gsa_fwd_workspace": (_sz, [_i] * 8),
    "gsa_fwd": (_i, [_vp] * 11 + [_i] * 8 + [_vp, _sz, _vp]),
    "gsa_bwd_workspace": (_sz, [_i] * 8),
    "gsa_bwd": (_i, [_vp] * 17 + [_i] * 8 + [_vp, _sz, _vp]),
    "gsa_recurrent_step": (_i, [_vp] * 8 + [_i] * 6 + [_vp]),
    "gla_device_error": (_i, [_vp, _i, ctypes.POINTER(_i)]),
    "gla_chunk_bwd_noalloc": (_i, [_vp] * 12 + [_i] * 7 + [_vp]),
    "gla_gate_logsigmoid": (_i, [_vp, _vp, ctypes.c_size_t, ctypes.c_float, _i, _vp]),
    "gla_gate_logsigmoid_bwd": (_i, [_vp, _vp, _vp, ctypes.c_size_t, ctypes.c_float, _i, _vp]),
    "gla_msgla_pool": (_i, [_vp, _vp] + [_i] * 6 + [_vp]),
    "gla_msgla_pool_bwd": (_i, [_vp, _vp] + [_i] * 6 + [_vp]),
    "gla_msgla_hold": (_i, [_vp, _vp] + [_i] * 6 + [_vp]),
    "gla_msgla_hold_bwd": (_i, [_vp, _vp] + [_i] * 6 + [_vp]),
    "gla_scan_fwd": (_i, [_vp] * 6 + [_i] * 6 + [_vp]),
    "gla_scan_bwd_workspace": (_sz, [_i] * 5),
    "gla_scan_bwd": (_i, [_vp] * 9 + [_i] * 6 + [_vp, _sz, _vp]),
    "gla_scan_step": (_i, [_vp] * 4 + [_i] * 5 + [_vp]),
    "gla_group_norm_fwd": (_i, [_vp] * 5 + [_i] * 7 + [ctypes.c_float, _i, _i, _vp]),
    "gla_group_norm_bwd_workspace": (_sz, [_i] * 7),
    "gla_group_norm_bwd": (_i, [_vp] * 9 + [_i] * 7 + [ctypes.c_float, _i, _i, _vp, _sz, _vp]),
    "gla_rotary": (_i, [_vp] * 6 + [ctypes.c_longlong] + [_i] * 7 + [ctypes.c_float] + [_i] * 5 + [_vp]),
}


class GLAError(RuntimeError):
    pass


def library_path() -> str:
    return os.path.join(_HERE, "lib", "libgla_b200.so")


def header_symbols(path: str = _HEADER):
    """Names of the functions declared in include/gla.h."""
    text = open(path).read()
    return re.findall(r"^\s*(?:const\s+char\s*\*|size_t|int)\s+(\w+)\s*\(", text, flags=re.M)


def load_library():
    """Load the CUDA library once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise GLAError(f"{path} is missing: build it with `python -m chunkwise_linear_rnn_02_b200.build_lib`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _LIB = lib
    return _LIB


def status_string(code: int) -> str:
    return load_library().gla_status_string(int(code)).decode()


def version() -> int:
    return load_library().gla_version()


def _check(code: int, what: str):
    if code != 0:
        raise GLAError(f"{what}: {status_string(code)}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise GLAError("tensors must be CUDA tensors: this library has no CPU path")
        if not t.is_contiguous():
            raise GLAError("tensors must be contiguous")


def _dtype_code(t):
    if t.dtype not in DTYPE_CODE:
        raise GLAError(f"unsupported dtype {t.dtype}; use torch.bfloat16 or torch.float32")
    return DTYPE_CODE[t.dtype]


def _state(t, shape, device):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape):
        raise GLAError(f"state tensors must be float32 of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    _need_cuda(t)
    return t


def workspace_bytes(kind: str, *args) -> int:
    lib = load_library()
    return int(getattr(lib, f"{kind}_workspace")(*[int(a) for a in args]))


def _workspace(nbytes: int, device):
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


# ------------------------------------------------------------------------------------------
def chunk_fwd(q, k, v, g, h0=None, chunk: int = 64, output_final_state: bool = True):
    """GLA forward: returns (o [B,H,T,dv], hT [B,H,dk,dv] fp32 or None)."""
    _need_cuda(q, k, v, g)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0 = _state(h0, (B, H, dk, dv), dev)
    o = torch.empty(B, H, T, dv, dtype=q.dtype, device=dev)
    hT = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if output_final_state else None
    ws, nb = _workspace(lib.gla_chunk_fwd_workspace(B, H, T, dk, dv, chunk, dt), dev)
    _check(lib.gla_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(o), _ptr(hT),
                             B, H, T, dk, dv, chunk, dt, _ptr(ws), nb, _stream(dev)), "gla_chunk_fwd")
    return o, hT


def chunk_bwd(q, k, v, g, do, h0=None, dhT=None, chunk: int = 64, need_dh0: bool = True):
    """GLA backward: returns (dq, dk, dv, dg, dh0 or None)."""
    _need_cuda(q, k, v, g, do)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0 = _state(h0, (B, H, dk, dv), dev)
    dhT = _state(dhT, (B, H, dk, dv), dev)
    dq, dkk, dg = (torch.empty_like(q) for _ in range(3))
    dvv = torch.empty_like(v)
    dh0 = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if need_dh0 else None
    ws, nb = _workspace(lib.gla_chunk_bwd_workspace(B, H, T, dk, dv, chunk, dt), dev)
    _check(lib.gla_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(do), _ptr(dhT),
                             _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dg), _ptr(dh0), B, H, T, dk, dv, chunk, dt,
                             _ptr(ws), nb, _stream(dev)), "gla_chunk_bwd")
    return dq, dkk, dvv, dg, dh0


def chunk_fwd_logit(q, k, v, x, tau: float, h0=None, chunk: int = 64, output_final_state: bool = True):
    """GLA forward from raw gate logits x (g = logsigmoid(x) / tau formed inside the kernels)."""
    _need_cuda(q, k, v, x)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0 = _state(h0, (B, H, dk, dv), dev)
    o = torch.empty(B, H, T, dv, dtype=q.dtype, device=dev)
    hT = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if output_final_state else None
    ws, nb = _workspace(lib.gla_chunk_fwd_logit_workspace(B, H, T, dk, dv, chunk, dt), dev)
    _check(lib.gla_chunk_fwd_logit(_ptr(q), _ptr(k), _ptr(v), _ptr(x), float(tau), _ptr(h0), _ptr(o), _ptr(hT),
                                   B, H, T, dk, dv, chunk, dt, _ptr(ws), nb, _stream(dev)), "gla_chunk_fwd_logit")
    return o, hT


def chunk_bwd_logit(q, k, v, x, tau: float, do, h0=None, dhT=None, chunk: int = 64, need_dh0: bool = True):
    """Backward of chunk_fwd_logit: returns (dq, dk, dv, dx, dh0 or None)."""
    _need_cuda(q, k, v, x, do)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0 = _state(h0, (B, H, dk, dv), dev)
    dhT = _state(dhT, (B, H, dk, dv), dev)
    dq, dkk, dx = (torch.empty_like(q) for _ in range(3))
    dvv = torch.empty_like(v)
    dh0 = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if need_dh0 else None
    ws, nb = _workspace(lib.gla_chunk_bwd_logit_workspace(B, H, T, dk, dv, chunk, dt), dev)
    _check(lib.gla_chunk_bwd_logit(_ptr(q), _ptr(k), _ptr(v), _ptr(x), float(tau), _ptr(h0), _ptr(do), _ptr(dhT),
                                   _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dx), _ptr(dh0), B, H, T, dk, dv, chunk, dt,
                                   _ptr(ws), nb, _stream(dev)), "gla_chunk_bwd_logit")
    return dq, dkk, dvv, dx, dh0


def recurrent_step(q, k, v, g, S):
    """One decode step; q, k, g [B,H,dk], v [B,H,dv]; S [B,H,dk,dv] fp32 updated in place.  Returns o."""
    _need_cuda(q, k, v, g, S)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _state(S, (B, H, dk, dv), q.device)
    o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check(load_library().gla_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S), _ptr(o), B, H, dk, dv,
                                             _dtype_code(q), _stream(q.device)), "gla_recurrent_step")
    return o


def gsa_fwd(q, k, v, phi, g, h0_1=None, h0_2=None, chunk: int = 64, save_p: bool = False,
            output_final_state: bool = True):
    """GSA forward: returns (o, p or None, hT1 or None, hT2 or None)."""
    _need_cuda(q, k, v, phi, g)
    B, H, T, dk = q.shape
    dv, m = v.shape[-1], phi.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0_1 = _state(h0_1, (B, H, dk, m), dev)
    h0_2 = _state(h0_2, (B, H, m, dv), dev)
    o = torch.empty(B, H, T, dv, dtype=q.dtype, device=dev)
    p = torch.empty(B, H, T, m, dtype=q.dtype, device=dev) if save_p else None
    hT1 = torch.empty(B, H, dk, m, dtype=torch.float32, device=dev) if output_final_state else None
    hT2 = torch.empty(B, H, m, dv, dtype=torch.float32, device=dev) if output_final_state else None
    ws, nb = _workspace(lib.gsa_fwd_workspace(B, H, T, dk, dv, m, chunk, dt), dev)
    _check(lib.gsa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(phi), _ptr(g), _ptr(h0_1), _ptr(h0_2), _ptr(o), _ptr(p),
                       _ptr(hT1), _ptr(hT2), B, H, T, dk, dv, m, chunk, dt, _ptr(ws), nb, _stream(dev)), "gsa_fwd")
    return o, p, hT1, hT2


def gsa_bwd(q, k, v, phi, g, do, h0_1=None, h0_2=None, dhT1=None, dhT2=None, chunk: int = 64,
            need_dh0: bool = True):
    """GSA backward: returns (dq, dk, dv, dphi, dg, dh0_1, dh0_2)."""
    _need_cuda(q, k, v, phi, g, do)
    B, H, T, dk = q.shape
    dv, m = v.shape[-1], phi.shape[-1]
    dt = _dtype_code(q)
    lib = load_library()
    dev = q.device
    h0_1 = _state(h0_1, (B, H, dk, m), dev)
    h0_2 = _state(h0_2, (B, H, m, dv), dev)
    dhT1 = _state(dhT1, (B, H, dk, m), dev)
    dhT2 = _state(dhT2, (B, H, m, dv), dev)
    dq, dkk = torch.empty_like(q), torch.empty_like(k)
    dvv, dphi, dg = torch.empty_like(v), torch.empty_like(phi), torch.empty_like(g)
    dh01 = torch.empty(B, H, dk, m, dtype=torch.float32, device=dev) if need_dh0 else None
    dh02 = torch.empty(B, H, m, dv, dtype=torch.float32, device=dev) if need_dh0 else None
    ws, nb = _workspace(lib.gsa_bwd_workspace(B, H, T, dk, dv, m, chunk, dt), dev)
    _check(lib.gsa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(phi), _ptr(g), _ptr(h0_1), _ptr(h0_2), _ptr(do),
                       _ptr(dhT1), _ptr(dhT2), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dphi), _ptr(dg), _ptr(dh01),
                       _ptr(dh02), B, H, T, dk, dv, m, chunk, dt, _ptr(ws), nb, _stream(dev)), "gsa_bwd")
    return dq, dkk, dvv, dphi, dg, dh01, dh02


def gsa_recurrent_step(q, k, v, phi, g, S1, S2):
    """One GSA decode step; S1 [B,H,dk,m], S2 [B,H,m,dv] fp32 updated in place.  Returns o [B,H,dv]."""
    _need_cuda(q, k, v, phi, g, S1, S2)
    B, H, dk = q.shape
    dv, m = v.shape[-1], phi.shape[-1]
    _state(S1, (B, H, dk, m), q.device)
    _state(S2, (B, H, m, dv), q.device)
    o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check(load_library().gsa_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(phi), _ptr(g), _ptr(S1), _ptr(S2),
                                             _ptr(o), B, H, dk, dv, m, _dtype_code(q), _stream(q.device)),
           "gsa_recurrent_step")
    return o


def device_error(reset: bool = True, device=None) -> int:
    """Synchronise the current stream and return the device error latch (0 = no error)."""
    code = ctypes.c_int(0)
    dev = device or torch.device("cuda", torch.cuda.current_device())
    _check(load_library().gla_device_error(_stream(dev), int(reset), ctypes.byref(code)), "gla_device_error")
    return code.value


# ------------------------------------------------------------------------------------------
def gate_logsigmoid(x, tau: float):
    """Raw-logit gate: g = logsigmoid(x) / tau (same shape and dtype as x)."""
    _need_cuda(x)
    g = torch.empty_like(x)
    _check(load_library().gla_gate_logsigmoid(_ptr(x), _ptr(g), x.numel(), float(tau), _dtype_code(x),
                                             _stream(x.device)), "gla_gate_logsigmoid")
    return g


def gate_logsigmoid_bwd(x, dg, tau: float):
    """dx = dg * sigmoid(-x) / tau."""
    _need_cuda(x, dg)
    dx = torch.empty_like(x)
    _check(load_library().gla_gate_logsigmoid_bwd(_ptr(x), _ptr(dg), _ptr(dx), x.numel(), float(tau),
                                                 _dtype_code(x), _stream(x.device)), "gla_gate_logsigmoid_bwd")
    return dx


def _msgla(name, inp, rows_out, T, s):
    _need_cuda(inp)
    B, H, _, D = inp.shape
    out = torch.empty(B, H, rows_out, D, dtype=inp.dtype, device=inp.device)
    _check(getattr(load_library(), name)(_ptr(inp), _ptr(out), B, H, T, D, int(s), _dtype_code(inp),
                                         _stream(inp.device)), name)
    return out


def msgla_pool(x, s: int):
    """Average pooling of non-overlapping blocks of s tokens: [B,H,T,D] -> [B,H,ceil(T/s),D]."""
    T = x.shape[2]
    return _msgla("gla_msgla_pool", x, -(-T // s), T, s)


def msgla_pool_bwd(dy, T: int, s: int):
    return _msgla("gla_msgla_pool_bwd", dy, T, T, s)


def msgla_hold(y, T: int, s: int):
    """Causal hold back to T tokens: token t gets pooled row (t+1)//s - 1 (zeros before that)."""
    return _msgla("gla_msgla_hold", y, T, T, s)


def msgla_hold_bwd(dout, s: int):
    T = dout.shape[2]
    return _msgla("gla_msgla_hold_bwd", dout, -(-T // s), T, s)


# ------------------------------------------------------------------------------------------
# Operators around the recurrences: the elementwise scan, the norm behind them, rotary positions.
# The calls below are a few microseconds of work for one decoded token, so the checks take the short way first.
def _operand(name, t, dtype, shape, device):
    """Address of a tensor that has to be a contiguous CUDA tensor of this dtype, shape and device; None stays."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise GLAError("tensors must be CUDA tensors: this library has no CPU path")
    if t.dtype is not dtype or t.shape != shape:
        raise GLAError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise GLAError(f"{name} is on {t.device}, the call runs on {device}: tensors must be on one device")
    raise GLAError("tensors must be contiguous")


def _first(t, rank):
    """Check the tensor that fixes dtype, shape and device; returns (dtype code, device)."""
    if not t.is_cuda:
        raise GLAError("tensors must be CUDA tensors: this library has no CPU path")
    if t.dim() != rank:
        raise GLAError(f"expected a tensor of {rank} dimensions, got shape {tuple(t.shape)}")
    return _dtype_code(t), t.device


def _too_long(t):
    """What to raise for a dimension of 2^31 or more: the library takes 32-bit sizes, and ctypes would drop the rest."""
    return GLAError(f"every dimension has to be below 2^31, got shape {tuple(t.shape)}")


# The current stream's handle without building a Stream object, where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _enqueue(name, device, *args):
    """Call an entry point on the current stream of the tensors' device, which need not be the current one."""
    fn = getattr(_LIB or load_library(), name)
    i = device.index
    if torch.cuda.current_device() == i:
        code = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            code = fn(*args, _raw_stream(i))
    if code != 0:
        raise GLAError(f"{name}: {status_string(code)}")


@functools.lru_cache(maxsize=256)
def _bytes(query, *sizes):
    return getattr(load_library(), query)(*sizes)


def _address(t):
    return None if t is None else t.data_ptr()


SCAN_KEEP = 64  # tokens between the states that scan_fwd(save_states=True) keeps


def scan_fwd(g, x, h0=None, complement: bool = False, output_final_state: bool = True, save_states: bool = False):
    """Elementwise scan h_t = exp(g_t) h_{t-1} + b_t, b = x or, complement, (1 - exp g) x, over [B,H,T,D].

    Returns (o [B,H,T,D], hT [B,H,D] fp32 or None, hc [B,H,ceil(T/64),D] fp32 or None); hc, the states before
    tokens 0, 64, ..., is what scan_bwd wants.  A [B,T,C] tensor goes in as [B,1,T,C].
    """
    dt, dev = _first(g, 4)
    B, H, T, D = g.shape
    if (B | H | T | D) >> 31:
        raise _too_long(g)
    gp, xp = _operand("g", g, g.dtype, g.shape, dev), _operand("x", x, g.dtype, g.shape, dev)
    hp = _operand("h0", h0, torch.float32, (B, H, D), dev)
    o = torch.empty_like(g)
    hT = g.new_empty((B, H, D), dtype=torch.float32) if output_final_state else None
    hc = g.new_empty((B, H, -(-T // SCAN_KEEP), D), dtype=torch.float32) if save_states else None
    _enqueue("gla_scan_fwd", dev, gp, xp, hp, o.data_ptr(), _address(hT), _address(hc), B, H, T, D, complement, dt)
    return o, hT, hc


def scan_bwd(g, x, do, h0=None, dhT=None, hc=None, complement: bool = False, need_dh0: bool = True):
    """Backward of scan_fwd: returns (dg, dx, dh0 or None).  Without hc the states are recomputed from h0."""
    dt, dev = _first(g, 4)
    B, H, T, D = g.shape
    if (B | H | T | D) >> 31:
        raise _too_long(g)
    gp, xp = _operand("g", g, g.dtype, g.shape, dev), _operand("x", x, g.dtype, g.shape, dev)
    dop = _operand("do", do, g.dtype, g.shape, dev)
    hp = _operand("h0", h0, torch.float32, (B, H, D), dev)
    dhp = _operand("dhT", dhT, torch.float32, (B, H, D), dev)
    hcp = _operand("hc", hc, torch.float32, (B, H, -(-T // SCAN_KEEP), D), dev)
    dg, dx = torch.empty_like(g), torch.empty_like(g)
    dh0 = g.new_empty((B, H, D), dtype=torch.float32) if need_dh0 else None
    ws, nb = (None, 0)
    if hc is None:
        ws, nb = _workspace(_bytes("gla_scan_bwd_workspace", B, H, T, D, 0), dev)
    _enqueue("gla_scan_bwd", dev, gp, xp, hp, hcp, dop, dhp, dg.data_ptr(), dx.data_ptr(), _address(dh0), B, H, T, D,
             complement, dt, _address(ws), nb)
    return dg, dx, dh0


def scan_step(g, x, S, complement: bool = False):
    """One token of scan_fwd: g, x [B,H,D]; S [B,H,D] fp32 updated in place.  Returns o [B,H,D]."""
    dt, dev = _first(g, 3)
    B, H, D = g.shape
    if (B | H | D) >> 31:
        raise _too_long(g)
    gp, xp = _operand("g", g, g.dtype, g.shape, dev), _operand("x", x, g.dtype, g.shape, dev)
    if S is None:
        raise GLAError("scan_step needs the state S")
    Sp = _operand("S", S, torch.float32, g.shape, dev)
    o = torch.empty_like(g)
    _enqueue("gla_scan_step", dev, gp, xp, Sp, o.data_ptr(), B, H, D, complement, dt)
    return o


_LAYOUTS = {"bhtd": 0, "bthd": 1}
_NORM_KINDS = {"group": 0, "rms": 1}
_ACTS = {"none": 0, "silu": 1, "sigmoid": 2}


def _choice(name, value, table):
    if value not in table:
        raise GLAError(f"{name} must be one of {', '.join(table)}; got {value!r}")
    return table[value]


def _norm_args(x, z, w, b, kind, act, layout):
    """Checks; returns dtype code, device, shape of y, weight rows, the pointers, and the codes behind them."""
    dt, dev = _first(x, 4)
    lay = _choice("layout", layout, _LAYOUTS)
    B, H, T, D = x.shape
    if (B | H | T | D) >> 31:
        raise _too_long(x)
    if lay:
        H, T = T, H
    out = (B, T, H, D)
    p = b if b is not None else w
    rows = H if p is None else p.shape[0] if p.dim() == 2 else -1
    if rows != 1 and rows != H:
        raise GLAError(f"w and b must be [H, D] or [1, D] with H = {H}")
    f32, wshape = torch.float32, (rows, D)
    return (dt, dev, out, rows, _operand("x", x, x.dtype, x.shape, dev), _operand("z", z, x.dtype, out, dev),
            _operand("w", w, f32, wshape, dev), _operand("b", b, f32, wshape, dev),
            _choice("kind", kind, _NORM_KINDS), _choice("act", act, _ACTS), lay)


def group_norm_fwd(x, z=None, w=None, b=None, kind: str = "group", act: str = "silu", eps: float = 1e-5,
                   layout: str = "bhtd"):
    """Norm of every head of a token, scaled and gated: y = (norm(x) * w + b) * act(z), or act(norm(x) * w + b)
    without z.

    x [B,H,T,D] (layout "bhtd", what the recurrences return) or [B,T,H,D] ("bthd"); z and the result are
    [B,T,H,D], that is, channels last.  w, b: fp32 [H,D], or [1,D] shared by the heads.  kind: "group" (mean and
    variance) or "rms"; act: "none", "silu", "sigmoid".
    """
    dt, dev, out, rows, xp, zp, wp, bp, kind, act, lay = _norm_args(x, z, w, b, kind, act, layout)
    B, T, H, D = out
    y = x.new_empty(out) if z is None else torch.empty_like(z)
    _enqueue("gla_group_norm_fwd", dev, xp, zp, wp, bp, y.data_ptr(), B, H, T, D, rows, kind, act, eps, lay, dt)
    return y


def group_norm_bwd(x, dy, z=None, w=None, b=None, kind: str = "group", act: str = "silu", eps: float = 1e-5,
                   layout: str = "bhtd"):
    """Backward of group_norm_fwd: returns (dx in x's layout, dz or None, dw or None, db or None)."""
    dt, dev, out, rows, xp, zp, wp, bp, kind, act, lay = _norm_args(x, z, w, b, kind, act, layout)
    B, T, H, D = out
    dyp = _operand("dy", dy, x.dtype, out, dev)
    dx = torch.empty_like(x)
    dz = None if z is None else torch.empty_like(z)
    dw = None if w is None else torch.empty_like(w)
    db = None if b is None else torch.empty_like(b)
    ws, nb = _workspace(_bytes("gla_group_norm_bwd_workspace", B, H, T, D, rows, w is not None, b is not None), dev)
    _enqueue("gla_group_norm_bwd", dev, xp, zp, wp, bp, dyp, dx.data_ptr(), _address(dz), _address(dw), _address(db),
             B, H, T, D, rows, kind, act, eps, lay, dt, _address(ws), nb)
    return dx, dz, dw, db


def rotary_frequencies(R: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       trained: int = 0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """Frequencies for rotary (radians a position, float64 [R/2]) and the scale of the rotated channels.

    freq_i = base^(-2i/R), changed for positions beyond the `trained` length by `factor`:
      "none"    as it is
      "linear"  freq / factor: positions are interpolated
      "ntk"     base * factor^(R/(R-2)): the slowest pair is interpolated, the fastest left alone
      "yarn"    pairs that turn more than `fast` times over the trained length are left alone, those that turn
                less than `slow` times are interpolated, a ramp in between; scale = 0.1 ln(factor) + 1
                ("YaRN: Efficient Context Window Extension of Large Language Models")
    Returns (freq, scale).  Made once for a model; the calls take them as they are.
    """
    if R < 2 or R % 2 or not base > 1 or not factor >= 1:
        raise GLAError(f"rotary_frequencies: needs an even R >= 2, base > 1 and factor >= 1; got {R}, {base}, {factor}")
    i = torch.arange(0, R, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        if R <= 2:
            raise GLAError("rotary_frequencies: ntk scaling needs R > 2")
        base = base * factor ** (R / (R - 2))
    freq = base ** (-i / R)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if trained <= 0 or not 0 < slow < fast:
            raise GLAError("rotary_frequencies: yarn scaling needs the trained length and 0 < slow < fast")

        def pair(turns):  # the (fractional) pair that turns so often over the trained length
            return R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(0, math.floor(pair(fast))), min(R - 1, math.ceil(pair(slow)))
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        ramp[i / 2 >= hi] = 1.0  # also where hi <= 0: every pair turns less than `slow` times
        freq = freq * (1 - ramp) + freq / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise GLAError(f"scaling must be one of none, linear, ntk, yarn; got {scaling!r}")
    return freq.to(device), scale


def _rotary(q, k, freq, pos, pos0, interleaved, scale, inverse, in_layout, out_layout):
    dt, dev = _first(q, 4)
    lin, lout = _choice("layout", in_layout, _LAYOUTS), _choice("out_layout", out_layout, _LAYOUTS)
    dtype = q.dtype
    B, Hq, T, D = q.shape
    if (B | Hq | T | D) >> 31:
        raise _too_long(q)
    if lin:
        Hq, T = T, Hq
    qp, kp, Hk, ko = _operand("q", q, dtype, q.shape, dev), None, 0, None
    if k is not None:
        if k.dim() != 4:
            raise GLAError(f"k must have 4 dimensions, got shape {tuple(k.shape)}")
        Hk = k.shape[2 if lin else 1]
        if Hk >> 31:
            raise _too_long(k)
        kp = _operand("k", k, dtype, (B, T, Hk, D) if lin else (B, Hk, T, D), dev)
    if not -(1 << 63) <= pos0 < 1 << 63:
        raise GLAError(f"pos0 has to fit 64 bits, got {pos0}")
    if freq.dim() != 1:
        raise GLAError(f"freq must be [R/2], got shape {tuple(freq.shape)}")
    if 2 * freq.shape[0] > D:
        raise GLAError(f"freq must have at most D/2 = {D // 2} frequencies, got {freq.shape[0]}")
    fp, pp, rows = _operand("freq", freq, torch.float64, freq.shape, dev), None, 0
    if pos is not None:
        one = pos.dim() == 1
        rows = 1 if one else B
        pp = _operand("pos", pos, torch.int64, (T,) if one else (B, T), dev)
    if lin == lout:
        qo = torch.empty_like(q)
        if k is not None:
            ko = torch.empty_like(k)
    else:
        qo = q.new_empty((B, T, Hq, D) if lout else (B, Hq, T, D))
        if k is not None:
            ko = k.new_empty((B, T, Hk, D) if lout else (B, Hk, T, D))
    _enqueue("gla_rotary", dev, qp, kp, qo.data_ptr(), _address(ko), fp, pp, pos0, rows, B, Hq, Hk, T, D,
             2 * freq.shape[0], scale, interleaved, inverse, lin, lout, dt)
    return qo, ko


def rotary(q, k, freq, pos=None, pos0: int = 0, interleaved: bool = False, scale: float = 1.0, layout: str = "bhtd",
           out_layout: str = "bhtd"):
    """Rotary positions of q and k (k may be None): returns (q', k') in out_layout.

    q [B,Hq,T,D], k [B,Hk,T,D] (layout "bhtd") or [B,T,H,D] ("bthd").  freq: float64 [R/2], radians a position for
    the pairs of the first R channels (rotary_frequencies).  Positions are pos0 + t, or pos0 + pos with pos int64
    [T] or [B,T].  Pairs are (i, i + R/2), or (2i, 2i+1) when interleaved; channels from R on are copied.
    """
    return _rotary(q, k, freq, pos, pos0, interleaved, scale, False, layout, out_layout)


def rotary_bwd(dq, dk, freq, pos=None, pos0: int = 0, interleaved: bool = False, scale: float = 1.0,
               layout: str = "bhtd", out_layout: str = "bhtd"):
    """Backward of rotary, called with the forward's arguments: dq, dk come in out_layout, the result in layout."""
    return _rotary(dq, dk, freq, pos, pos0, interleaved, scale, True, out_layout, layout)
