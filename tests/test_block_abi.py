"""CPU tests of the block entry points: every argument error is caught on the host, with its status, before anything
is launched."""
import ctypes
import os

import pytest

import calibration_free_w4a4_amd as orbq

pytestmark = pytest.mark.skipif(not os.path.exists(orbq.library_path()), reason="liborbq.so not built")
P = 0x10000   # an aligned dummy device address; the host never reads it
OK, ARG, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
NONE, LAYER, RMS = 0, 1, 2
F32, BF16, F16 = 0, 1, 2


class Norms(ctypes.Structure):
    """orbq_norms as include/orbq.h declares it."""
    _fields_ = [("norm", ctypes.c_int), ("post", ctypes.c_int), ("eps", ctypes.c_float), ("post_eps", ctypes.c_float)] + \
        [(a, ctypes.c_void_p) for a in ("weight", "post_weight", "gate", "scale", "shift")] + \
        [(a, ctypes.c_int64) for a in ("gate_ld", "scale_ld", "shift_ld")] + \
        [("weight_type", ctypes.c_int), ("mod_type", ctypes.c_int), ("cu", ctypes.c_void_p), ("groups", ctypes.c_int32)]


class Grads(ctypes.Structure):
    _fields_ = [(a, ctypes.c_void_p) for a in ("gate", "scale", "shift")] + \
        [(a, ctypes.c_int64) for a in ("gate_ld", "scale_ld", "shift_ld")] + [("weight", ctypes.c_void_p), ("post_weight", ctypes.c_void_p)]


def norms(**kw):
    f = dict(norm=LAYER, post=NONE, eps=1e-6, post_eps=1e-6, gate=P, scale=P, shift=P, gate_ld=64, scale_ld=64, shift_ld=64,
             weight_type=F32, mod_type=F32, groups=2)
    f.update(kw)
    return Norms(**f)


def test_the_binding_packs_the_structs_as_declared():
    from calibration_free_w4a4_amd import block
    assert block._NORMS.size == ctypes.sizeof(Norms) and block._GRADS.size == ctypes.sizeof(Grads)
    values = (1, 2, 0.5, 0.25, 3, 4, 5, 6, 7, 8, 9, 10, 1, 2, 1 << 40, 12)
    got = Norms.from_buffer_copy(block._NORMS.pack(*values))
    assert tuple(getattr(got, f[0]) for f in Norms._fields_) == values
    got = Grads.from_buffer_copy(block._GRADS.pack(*range(1, 9)))
    assert [getattr(got, f[0]) for f in Grads._fields_] == list(range(1, 9))


def forward(p=None, n=8, d=64, x=P, xld=64, y=P, yld=64, r=P, rld=64, h=P, hld=64, st=BF16, br=BF16):
    p = None if p == "null" else ctypes.byref(norms(**(p or {})))
    return orbq.load().orbq_block_norm(p, n, d, x, xld, y, yld, r, rld, h, hld, st, br, None)


COMMON = [
    (dict(p="null"), ARG), (dict(p=dict(norm=3)), ARG), (dict(p=dict(post=-1)), ARG), (dict(st=5), ARG), (dict(br=-1), ARG),
    (dict(p=dict(weight_type=9)), ARG), (dict(p=dict(mod_type=9)), ARG), (dict(st=BF16, br=F16), UNSUPPORTED),
    (dict(st=F16, br=F32), UNSUPPORTED), (dict(n=-1), ARG), (dict(d=0), ARG), (dict(d=16385), UNSUPPORTED),
    (dict(n=(1 << 30) + 2), UNSUPPORTED), (dict(p=dict(groups=0)), ARG), (dict(p=dict(groups=3)), ARG),
    (dict(p=dict(cu=P + 2)), ALIGN), (dict(p=dict(eps=-1.0)), ARG), (dict(p=dict(eps=float("nan"))), ARG),
    (dict(p=dict(post_eps=float("inf"))), ARG), (dict(p=dict(norm=NONE)), ARG), (dict(p=dict(post_weight=P)), ARG),
    (dict(y=None), ARG), (dict(p=dict(gate_ld=-1)), ARG), (dict(p=dict(scale=P + 2)), ALIGN),
    (dict(p=dict(weight=P + 1, weight_type=BF16)), ALIGN), (dict(y=P + 1), ALIGN), (dict(yld=-64), ARG)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(x=None), ARG), (dict(h=None), ARG), (dict(p=dict(norm=NONE, scale=None, shift=None)), ARG),
    (dict(p=dict(norm=NONE, scale=None, shift=None), h=None, r=None), ARG), (dict(rld=63), ARG), (dict(hld=0), ARG),
    (dict(x=P + 1), ALIGN), (dict(r=P + 1), ALIGN), (dict(h=P + 2, st=F32, br=F32), ALIGN),
    (dict(n=0, x=None, r=None, h=None), OK)])
def test_forward(kw, want):
    assert forward(**kw) == want, orbq.load().orbq_last_error().decode()


def backward(p=None, n=8, d=64, r=P, rld=64, y=P, yld=64, dr=P, drld=64, dh=P, dhld=64, dx=P, dxld=64, dy=P, dyld=64, g=None,
             st=BF16, br=BF16, ws=P, ws_bytes=1 << 30):
    p = None if p == "null" else ctypes.byref(norms(**(p or {})))
    g = None if g == "null" else ctypes.byref(Grads(**(g or dict(gate=P, gate_ld=64))))
    return orbq.load().orbq_block_norm_backward(p, n, d, r, rld, y, yld, dr, drld, dh, dhld, dx, dxld, dy, dyld, g, st, br, ws,
                                                ws_bytes, None)


PLAIN = dict(norm=NONE, scale=None, shift=None)


@pytest.mark.parametrize("kw,want", [(dict(kw, g="null"), w) for kw, w in COMMON] + [
    (dict(r=None), ARG), (dict(dh=None), ARG), (dict(p=PLAIN), ARG), (dict(p=PLAIN, dh=None, dr=None), ARG),
    (dict(p=PLAIN, dh=None, g=dict(scale=P, scale_ld=64)), ARG), (dict(p=PLAIN, dh=None, g=dict(weight=P)), ARG),
    (dict(g=dict(post_weight=P)), ARG), (dict(p=dict(gate=None), y=None, dy=P, g="null"), ARG),
    (dict(p=dict(gate=None), y=None, dy=None), ARG), (dict(g=dict(gate=P, gate_ld=63)), ARG), (dict(g=dict(shift=P + 2)), ALIGN),
    (dict(dxld=63), ARG), (dict(dyld=0), ARG), (dict(dx=P + 1), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(ws=P + 8), ALIGN), (dict(n=0, r=None, dr=None, dh=None, dx=None, dy=None, g="null"), OK),
    (dict(dx=None, dy=None, g="null"), OK)])
def test_backward(kw, want):
    assert backward(**kw) == want, orbq.load().orbq_last_error().decode()


def test_workspace_bytes():
    f = orbq.load().orbq_block_norm_backward_workspace_bytes
    assert f(0, 64, 1) == 3 * 64 * 4 and f(1, 64, 1) == 3 * 64 * 4
    assert f(1000, 64, 5) == f(1000, 64, 1) + 4 * 3 * 64 * 4           # a place more for each group
    assert f(10 ** 6, 64, 1) < 5000 * 3 * 64 * 4                      # chunks go by the card, not by the rows
    assert f(-1, 64, 1) == f(1, 0, 1) == f(1, 16385, 1) == f(1, 64, 0) == 0
