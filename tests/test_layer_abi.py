"""Refusals of the scan, group-norm and rotary entry points (no GPU needed): every call here fails a
check, or has nothing to do, before any launch."""
import ctypes

import pytest
import torch

from chunkwise_linear_rnn_02_b200 import binding
from chunkwise_linear_rnn_02_b200.build_lib import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 0x7F0000000000  # a 256-byte aligned fake device address: never dereferenced by these tests
ODD = P + 1         # not aligned to any element type


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


def _call(fn, defaults, **change):
    args = dict(defaults, **change)
    assert set(args) == set(defaults)
    return fn(*args.values())


SCAN_FWD = dict(g=P, x=P, h0=None, o=P, hT=None, hc=None, B=1, H=1, T=8, D=16, input=0, dtype=1, stream=None)
SCAN_BWD = dict(g=P, x=P, h0=None, hc=None, dO=P, dhT=None, dg=P, dx=P, dh0=None, B=1, H=1, T=8, D=16, input=0,
                dtype=1, ws=P, nb=1 << 40, stream=None)
SCAN_STEP = dict(g=P, x=P, S=P, o=P, B=1, H=1, D=16, input=0, dtype=1, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(g=None), INVALID), (dict(x=None), INVALID), (dict(x=ODD), INVALID),
    (dict(B=0), INVALID), (dict(H=-1), INVALID), (dict(D=0), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(input=2), UNSUPPORTED), (dict(input=-1), UNSUPPORTED),
    (dict(B=1 << 20, H=1 << 10), UNSUPPORTED),
    (dict(B=1 << 16, H=1 << 16), INVALID), (dict(D=(1 << 31) - 1, B=2), UNSUPPORTED),
])
def test_scan_refusals(lib, change, code):
    assert _call(lib.gla_scan_fwd, SCAN_FWD, **change) == code
    assert _call(lib.gla_scan_bwd, SCAN_BWD, **change) == code
    assert _call(lib.gla_scan_step, SCAN_STEP, **change) == code


def test_scan_more_refusals(lib):
    assert _call(lib.gla_scan_fwd, SCAN_FWD, T=-1) == INVALID
    assert _call(lib.gla_scan_fwd, SCAN_FWD, o=None) == INVALID
    for name in ("h0", "hT", "hc"):
        assert _call(lib.gla_scan_fwd, SCAN_FWD, **{name: P + 2}) == INVALID  # fp32 on two bytes
    for name in ("dO", "dg", "dx"):
        assert _call(lib.gla_scan_bwd, SCAN_BWD, **{name: None}) == INVALID
    for name in ("h0", "hc", "dhT", "dh0"):
        assert _call(lib.gla_scan_bwd, SCAN_BWD, **{name: P + 2}) == INVALID
    assert _call(lib.gla_scan_step, SCAN_STEP, S=None) == INVALID
    assert _call(lib.gla_scan_step, SCAN_STEP, o=None) == INVALID
    # without kept states the backward recomputes them into the workspace
    need = lib.gla_scan_bwd_workspace(2, 3, 130, 40, 0)
    assert need >= 2 * 3 * 3 * 40 * 4 and need % 256 == 0
    assert lib.gla_scan_bwd_workspace(2, 3, 130, 40, 1) == 0
    assert lib.gla_scan_bwd_workspace(2, 3, 0, 40, 0) == 0
    assert lib.gla_scan_bwd_workspace(0, 3, 130, 40, 0) == 0
    size = dict(B=2, H=3, T=130, D=40)
    assert _call(lib.gla_scan_bwd, SCAN_BWD, ws=None, **size) == WORKSPACE
    assert _call(lib.gla_scan_bwd, SCAN_BWD, nb=need - 1, **size) == WORKSPACE
    assert _call(lib.gla_scan_bwd, SCAN_BWD, ws=P + 16, **size) == WORKSPACE


NORM = dict(x=P, z=P, w=P, b=P, y=P, B=1, H=4, T=8, D=16, rows=4, kind=0, act=1, eps=1e-5, layout=0, dtype=1, stream=None)
NORM_BWD = dict(x=P, z=P, w=P, b=P, dy=P, dx=P, dz=P, dw=P, db=P, B=1, H=4, T=8, D=16, rows=4, kind=0, act=1,
                eps=1e-5, layout=0, dtype=1, ws=P, nb=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(z=ODD), INVALID), (dict(w=P + 2), INVALID),
    (dict(b=P + 2), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID),
    (dict(rows=2), INVALID), (dict(rows=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(kind=2), UNSUPPORTED), (dict(act=3), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(D=8193), UNSUPPORTED), (dict(H=65536, rows=1), UNSUPPORTED), (dict(B=1 << 20, T=1 << 12), UNSUPPORTED),
])
def test_group_norm_refusals(lib, change, code):
    assert _call(lib.gla_group_norm_fwd, NORM, **change) == code
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, **change) == code


def test_group_norm_more_refusals(lib):
    assert _call(lib.gla_group_norm_fwd, NORM, y=None) == INVALID
    assert _call(lib.gla_group_norm_fwd, NORM, T=0, x=None, z=None, y=None) == OK  # nothing to do
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, dy=None) == INVALID
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, dx=None) == INVALID
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, z=None) == INVALID  # dz without z
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, dw=P + 2) == INVALID
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, T=0, dw=None, db=None) == OK
    need = lib.gla_group_norm_bwd_workspace(1, 4, 8, 16, 4, 1, 1)
    assert need > 0 and need % 512 == 0
    assert lib.gla_group_norm_bwd_workspace(1, 4, 8, 16, 4, 1, 0) == need // 2
    assert lib.gla_group_norm_bwd_workspace(1, 4, 8, 16, 4, 0, 0) == 0
    assert lib.gla_group_norm_bwd_workspace(1, 4, 8, 16, 3, 1, 1) == 0
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, ws=None) == WORKSPACE
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, nb=need - 1) == WORKSPACE
    assert _call(lib.gla_group_norm_bwd, NORM_BWD, ws=P + 16) == WORKSPACE


ROTARY = dict(q=P, k=P, qo=P + (1 << 20), ko=P + (1 << 21), freq=P, pos=P, pos0=0, pos_rows=1, B=2, Hq=4, Hk=2, T=8, D=16, R=8,
              scale=1.0, interleaved=0, inverse=0, in_layout=0, out_layout=0, dtype=1, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(q=ODD), INVALID), (dict(ko=ODD), INVALID), (dict(freq=None), INVALID), (dict(freq=P + 4), INVALID),
    (dict(pos=None), INVALID), (dict(pos=P + 4), INVALID), (dict(pos_rows=3), INVALID), (dict(pos_rows=-1), INVALID),
    (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID),
    (dict(R=0), INVALID), (dict(R=7), INVALID), (dict(R=18), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(in_layout=2), UNSUPPORTED), (dict(out_layout=-1), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(D=8194), UNSUPPORTED), (dict(B=1 << 20, T=1 << 12, pos_rows=1), UNSUPPORTED),
    (dict(out_layout=1, qo=P), INVALID), (dict(in_layout=1, ko=P), INVALID),  # in place only with equal layouts
    (dict(T=0, q=None, k=None, qo=None, ko=None, freq=None, pos=None), OK),
])
def test_rotary_refusals(lib, change, code):
    assert _call(lib.gla_rotary, ROTARY, **change) == code


def test_binding_refuses_cpu_tensors_and_bad_choices():
    x, s = torch.zeros(1, 2, 8, 8), torch.zeros(1, 2, 8)
    f = torch.zeros(4, dtype=torch.float64)
    for call in (lambda: binding.scan_fwd(x, x), lambda: binding.scan_bwd(x, x, x), lambda: binding.scan_step(s, s, s),
                 lambda: binding.group_norm_fwd(x), lambda: binding.group_norm_bwd(x, x),
                 lambda: binding.rotary(x, x, f), lambda: binding.rotary_bwd(x, None, f)):
        with pytest.raises(binding.GLAError, match="no CPU path"):
            call()
    assert ctypes.sizeof(ctypes.c_longlong) == 8
