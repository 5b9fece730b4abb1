"""The lapmix part of the C ABI without a GPU: exports, sizes and refusals.  Every call
here is refused, or is host arithmetic, before any device is touched."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import laplacian_nystr_approximation_amd as L
from laplacian_nystr_approximation_amd import lapmix as M
from laplacian_nystr_approximation_amd import lapnys as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30  # addresses a GiB apart; never dereferenced


def _scan(**kw):
    return L.make_scan_params(**{**dict(B=2, H=3, N=600, d=64, dtype="bf16"), **kw})


def _norm(**kw):
    return L.make_norm_params(**{**dict(B=2, H=3, N=10, d=64, x_dtype="f32", r_dtype="bf16", y_dtype="bf16"), **kw})


def _fwd(p, x=A, g=2 * A, h0=None, lengths=None, y=3 * A, hN=None, states=None, ws=16 * A, n=1 << 40):
    return L.library().lapmix_scan_forward_ws(x, g, h0, lengths, y, hN, states, ctypes.byref(p), ws, n, None)


def _bwd(p, x=A, g=2 * A, states=3 * A, lengths=None, dy=4 * A, dhN=None, dx=5 * A, dg=6 * A, dh0=None, ws=16 * A,
         n=1 << 40):
    return L.library().lapmix_scan_backward_ws(x, g, states, lengths, dy, dhN, dx, dg, dh0, ctypes.byref(p), ws, n,
                                               None)


def _step(p, x=A, g=2 * A, slots=None, h_in=3 * A, h_out=4 * A, n=2, y=5 * A):
    return L.library().lapmix_scan_step(x, g, slots, h_in, h_out, n, y, ctypes.byref(p), None)


def _nf(p, x=A, r=2 * A, w=3 * A, s=4 * A, y=5 * A, scale=None):
    return L.library().lapmix_norm_forward(x, r, w, s, y, scale, ctypes.byref(p), None)


def _nb(p, dy=A, s=2 * A, w=3 * A, ds=4 * A, dr=5 * A, dx=6 * A, dw=7 * A, ws=16 * A, n=1 << 40):
    return L.library().lapmix_norm_backward_ws(dy, s, w, ds, dr, dx, dw, ctypes.byref(p), ws, n, None)


def test_exports_are_what_the_header_declares():
    text = open(os.path.join(ROOT, "include", "lapmix.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(lapmix_[a-z0-9_]+)\s*\(", text))
    nm = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (lapmix_\w+)", nm)) == declared
    assert declared == {n for n in dir(M) if n.startswith("lapmix_") and not n.endswith("_params")}


def test_struct_layouts():
    assert ctypes.sizeof(M.lapmix_scan_params) == 6 * 4 + 9 * 8
    assert ctypes.sizeof(M.lapmix_norm_params) == 10 * 4 + 3 * 8


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), B.LAPNYS_ERR_INVALID_ARG), (dict(H=-1), B.LAPNYS_ERR_INVALID_ARG),
    (dict(N=0), B.LAPNYS_ERR_INVALID_ARG), (dict(d=0), B.LAPNYS_ERR_INVALID_ARG),
    (dict(dtype=2), B.LAPNYS_ERR_UNSUPPORTED), (dict(dtype=7), B.LAPNYS_ERR_UNSUPPORTED),
    (dict(B=1 << 16, H=1 << 16), B.LAPNYS_ERR_UNSUPPORTED), (dict(B=1 << 15, H=1 << 15, d=4), B.LAPNYS_ERR_UNSUPPORTED),
    (dict(B=1 << 14, H=1 << 8, d=65), B.LAPNYS_ERR_UNSUPPORTED), (dict(B=1, H=1, N=(1 << 30) + 1), B.LAPNYS_ERR_UNSUPPORTED),
])
def test_scan_params_refused(kw, code):
    p = _scan(**kw)
    n = ctypes.c_size_t(77)
    for f in (L.library().lapmix_scan_workspace_size, L.library().lapmix_scan_states_size):
        assert f(ctypes.byref(p), ctypes.byref(n)) == code and n.value == 77
    assert _fwd(p) == code and _bwd(p) == code and _step(p) == code


def test_scan_flags_and_null_params():
    p = _scan()
    p.flags = 4
    assert _fwd(p) == B.LAPNYS_ERR_INVALID_ARG
    assert L.library().lapmix_scan_forward_ws(A, 2 * A, None, None, 3 * A, None, None, None, None, 0, None) == \
        B.LAPNYS_ERR_INVALID_ARG
    assert L.library().lapmix_scan_workspace_size(ctypes.byref(_scan()), None) == B.LAPNYS_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        _scan(gate="tanh")


def test_scan_strides_refused():
    for name in ("x_stride", "g_stride", "y_stride"):
        p = _scan()
        getattr(p, name)[:] = (64 * 600 * 3, -64 * 600, 64)
        assert _fwd(p) == B.LAPNYS_ERR_INVALID_ARG, name
        getattr(p, name)[:] = (1 << 62, 64 * 600, 64)
        assert _fwd(p) == B.LAPNYS_ERR_INVALID_ARG, name
    # written elements that coincide: tokens on top of each other, heads inside a token's channels
    for st in ((64 * 600 * 3, 64 * 600, 0), (64 * 600 * 3, 32, 64 * 3), (64 * 600, 64 * 600, 64)):
        p = _scan()
        p.y_stride[:] = st
        assert _fwd(p) == B.LAPNYS_ERR_INVALID_ARG, st
        p = _scan()
        p.x_stride[:] = st
        assert _bwd(p) == B.LAPNYS_ERR_INVALID_ARG, st


def test_scan_buffers_refused():
    p = _scan()
    bad = B.LAPNYS_ERR_INVALID_ARG
    n = 2 * 3 * 600 * 64 * 2
    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(x=A + 1), dict(y=A), dict(y=2 * A + n - 2),
               dict(h0=3 * A), dict(hN=3 * A + 64), dict(hN=A), dict(h0=7 * A, hN=7 * A + 4), dict(hN=7 * A + 2),
               dict(states=3 * A), dict(states=7 * A, hN=7 * A), dict(states=7 * A, h0=7 * A),
               dict(lengths=3 * A), dict(lengths=7 * A + 1)):
        assert _fwd(p, **kw) == bad, kw
    for kw in (dict(states=None), dict(dy=None), dict(dx=None), dict(dg=None), dict(dx=A), dict(dg=2 * A),
               dict(dx=6 * A), dict(dx=4 * A), dict(dh0=5 * A), dict(dhN=5 * A), dict(dh0=3 * A), dict(dh0=4 * A),
               dict(dhN=7 * A, dh0=7 * A + 8)):
        assert _bwd(p, **kw) == bad, kw


def test_interleaved_gradients_are_told_from_overlapping_ones():
    """dx and dg as the halves of a [B, N, 2, H, d] buffer pass the overlap check (the call then
    stops at the missing workspace), a shifted pair does not."""
    p = _scan(N=640)
    st = (640 * 2 * 3 * 64, 64, 2 * 3 * 64)
    p.x_stride[:] = st
    p.g_stride[:] = st
    bad, stops = B.LAPNYS_ERR_INVALID_ARG, B.LAPNYS_ERR_WORKSPACE
    apart = 3 * 64 * 2
    assert L.lapmix_scan_workspace_size(p) > 0
    assert _bwd(p, dx=5 * A, dg=5 * A + apart - 2, ws=None) == bad
    assert _bwd(p, dx=5 * A, dg=5 * A + 64 * 2, ws=None) == bad  # the next head
    assert _bwd(p, dx=5 * A, dg=5 * A + 2 * apart, ws=None) == bad  # the next token
    assert _bwd(p, dx=5 * A, dg=5 * A + apart, ws=None) == stops
    assert _bwd(p, dx=5 * A, dg=5 * A - apart, ws=None) == stops
    # the same for the forward's inputs and output as three parts of one buffer
    q = _scan(N=640)
    for st in (q.x_stride, q.g_stride, q.y_stride):
        st[:] = (640 * 3 * 3 * 64, 64, 3 * 3 * 64)
    assert _fwd(q, x=A, g=A + apart, y=A + 2 * apart, ws=None) == stops
    assert _fwd(q, x=A, g=A + apart, y=A + apart, ws=None) == bad
    # the state carried in place stops at the workspace too
    assert _fwd(q, h0=7 * A, hN=7 * A, y=4 * A, ws=None) == stops
    assert _bwd(p, dhN=7 * A, dh0=7 * A, ws=None) == stops


def test_step_refusals():
    assert _step(_scan()) == B.LAPNYS_ERR_SHAPE
    p = _scan(N=1)
    bad = B.LAPNYS_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(h_in=None), dict(h_out=None), dict(n=0), dict(n=-1),
               dict(h_out=3 * A + 4), dict(y=3 * A), dict(y=4 * A), dict(slots=4 * A), dict(h_out=A)):
        assert _step(p, **kw) == bad, kw
    assert _step(p, n=1) == B.LAPNYS_ERR_SHAPE
    assert _step(_scan(B=(1 << 25) + 1, H=1, N=1, d=1), n=1 << 30) == B.LAPNYS_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), B.LAPNYS_ERR_INVALID_ARG), (dict(d=-4), B.LAPNYS_ERR_INVALID_ARG),
    (dict(eps=0.0), B.LAPNYS_ERR_INVALID_ARG), (dict(eps=float("nan")), B.LAPNYS_ERR_INVALID_ARG),
    (dict(eps=float("inf")), B.LAPNYS_ERR_INVALID_ARG), (dict(x_dtype=2), B.LAPNYS_ERR_UNSUPPORTED),
    (dict(r_dtype=2), B.LAPNYS_ERR_UNSUPPORTED), (dict(y_dtype=3), B.LAPNYS_ERR_UNSUPPORTED),
    (dict(group=64), B.LAPNYS_ERR_INVALID_ARG), (dict(H=257, d=64), B.LAPNYS_ERR_UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 16), B.LAPNYS_ERR_UNSUPPORTED),
])
def test_norm_params_refused(kw, code):
    p = _norm(**kw)
    n = ctypes.c_size_t(77)
    assert L.library().lapmix_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code and n.value == 77
    assert _nf(p) == code and _nb(p) == code


def test_norm_groups_refused():
    bad = B.LAPNYS_ERR_INVALID_ARG
    e = dict(y_dtype="e4m3")
    for group in (8, 24, 1024, -16):
        assert _nf(_norm(**e, group=group), scale=8 * A) == bad
    assert _nf(_norm(**e, group=128), scale=8 * A) == B.LAPNYS_ERR_SHAPE  # of 192 columns
    assert _nf(_norm(**e, group=64)) == bad  # no scales
    assert _nf(_norm(), scale=8 * A) == bad  # scales without e4m3
    # groups need 16-byte bases and strides
    assert _nf(_norm(**e, group=64), scale=8 * A, x=A + 4) == B.LAPNYS_ERR_UNSUPPORTED
    assert _nf(_norm(**e, group=64), scale=8 * A, r=2 * A + 2) == B.LAPNYS_ERR_UNSUPPORTED
    p = _norm(**e, group=64)
    p.x_stride[:] = (3 * 10 * 64 + 4, 640, 64)
    assert _nf(p, scale=8 * A) == B.LAPNYS_ERR_UNSUPPORTED
    # e4m3 has no backward of its own
    assert _nb(_norm(**e)) == B.LAPNYS_ERR_UNSUPPORTED


def test_norm_buffers_refused():
    bad = B.LAPNYS_ERR_INVALID_ARG
    p = _norm()
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(y=A), dict(s=A), dict(y=4 * A), dict(s=2 * A + 16),
               dict(y=2 * A), dict(w=3 * A + 2), dict(y=5 * A + 1), dict(s=3 * A)):
        assert _nf(p, **kw) == bad, kw
    for kw in (dict(dy=None), dict(s=None), dict(w=None), dict(dr=None, dx=None, dw=None), dict(dr=A), dict(dr=2 * A),
               dict(dx=2 * A), dict(dx=5 * A), dict(dw=3 * A), dict(dr=4 * A + 2), dict(dx=4 * A),
               dict(ds=5 * A, dx=5 * A)):
        assert _nb(p, **kw) == bad, kw
    need = L.lapmix_norm_workspace_size(p)
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=16 * A + 64)):
        assert _nb(p, **kw) == B.LAPNYS_ERR_WORKSPACE
    assert _nb(p, ws=5 * A) == bad
    p.reserved = 1
    assert _nf(p) == bad


def test_sizes():
    p = _scan()
    assert L.lapmix_scan_states_size(p) == 2 * 3 * -(-600 // L.LAPMIX_SCAN_TILE) * 64 * 4
    assert L.lapmix_scan_states_size(_scan(N=L.LAPMIX_SCAN_TILE)) == 2 * 3 * 64 * 4
    assert L.lapmix_scan_workspace_size(p) % 256 == 0
    assert L.lapmix_norm_workspace_size(_norm()) >= 192 * 4


def test_binding_checks_tensors():
    p = _scan(B=1, H=1, N=4, d=8)
    t = torch.zeros(1, 1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        L.lapmix_scan_forward_ws(t, t, t, p, None)
    with pytest.raises(ValueError, match="x: expected"):
        L.lapmix_scan_forward_ws(t.float(), t, t, p, None)
    with pytest.raises(ValueError, match="g: expected"):
        L.lapmix_scan_forward_ws(A, t[..., :7], t, p, None)
    with pytest.raises(ValueError, match="hN: expected"):
        L.lapmix_scan_forward_ws(A, 2 * A, 3 * A, p, None, hN=torch.zeros(7))
    with pytest.raises(ValueError, match="states: expected"):
        L.lapmix_scan_forward_ws(A, 2 * A, 3 * A, p, None, states=torch.zeros(7))
    with pytest.raises(ValueError, match="x: expected .*float16"):
        L.lapmix_scan_forward_ws(t.half(), t, t, p, None)
    with pytest.raises(ValueError, match="lengths: expected .*float32"):
        L.lapmix_scan_forward_ws(A, 2 * A, 3 * A, p, None, lengths=torch.zeros(1))
    with pytest.raises(ValueError, match="h0: expected .*int32"):
        L.lapmix_scan_forward_ws(A, 2 * A, 3 * A, p, None, h0=torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="n_slots"):
        L.lapmix_scan_step(A, 2 * A, 3 * A, 4 * A, 5 * A, _scan(N=1))
    with pytest.raises(ValueError, match="slots: expected"):
        L.lapmix_scan_step(A, 2 * A, 3 * A, 4 * A, 5 * A, _scan(N=1), slots=torch.zeros(2, dtype=torch.int64), n_slots=2)
    q = _norm(B=1, H=1, N=4, d=8)
    with pytest.raises(ValueError, match="w: expected"):
        L.lapmix_norm_forward(A, torch.zeros(8, dtype=torch.bfloat16), 3 * A, q)
    with pytest.raises(ValueError, match="dr: expected"):
        L.lapmix_norm_backward_ws(A, 2 * A, 3 * A, q, None, dr=torch.zeros(31, dtype=torch.bfloat16))
