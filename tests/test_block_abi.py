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


# ------------------------------------------------------------------------------------- kv_append_rope
def append(c=None, t=None, start=P, cu=P, total=6, most=3, r=None, pos=P, n_pos=6, q=None, qw=None, k=P, kt=256, kh=128, kw=None, v=P,
           vt=256, vh=128, eps=1e-6, dtype=1):
    from tests.test_attention_abi import Structs, cache, table
    c = None if c == "null" else ctypes.byref(cache(Structs, **(c or {})))
    t = None if t == "null" else ctypes.byref(table(Structs, **(t or {})))
    f = dict(axes=1, dims=(ctypes.c_int32 * 4)(128), freqs=P, layout=0)
    f.update({} if r == "null" else r or {})
    r = None if r == "null" else ctypes.byref(Structs._Rope(f["axes"], (ctypes.c_int32 * 4)(*f["dims"]), f["freqs"], f["layout"]))
    h = dict(x=P, y=P, heads=4, x_token=512, x_head=128, y_token=512, y_head=128)
    h.update({} if q == "null" else q or {})
    q = None if q == "null" else ctypes.byref(Structs._Heads(*h.values()))
    return orbq.load().orbq_kv_append_rope(c, t, start, cu, total, most, r, pos, n_pos, q, qw, k, kt, kh, kw, v, vt, vh, eps, dtype, None)


def test_kv_append_rope():
    from tests.test_attention_abi import CACHE_ERRORS
    for c, t, want in CACHE_ERRORS:
        assert append(c, t) == want, (c, t, orbq.load().orbq_last_error())
    for kw, want in ((dict(c="null"), ARG), (dict(t="null"), ARG), (dict(r="null"), ARG), (dict(r=dict(axes=5)), UNSUPPORTED),
                     (dict(r=dict(dims=(130, 0, 0, 0))), ARG), (dict(r=dict(dims=(33, 0, 0, 0))), ARG), (dict(r=dict(dims=(0, 0, 0, 0))), ARG),
                     (dict(r=dict(layout=3)), ARG), (dict(r=dict(freqs=None)), ARG), (dict(pos=None), ARG), (dict(pos=P + 2), ALIGN),
                     (dict(n_pos=0), ARG), (dict(n_pos=4), ARG), (dict(start=None), ARG), (dict(start=P + 2), ALIGN), (dict(cu=P + 1), ALIGN),
                     (dict(cu=None, total=5), ARG), (dict(total=-1), ARG), (dict(most=-1), ARG), (dict(total=1 << 31), UNSUPPORTED),
                     (dict(t=dict(batch=0)), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=P + 8), ALIGN), (dict(kt=260), ALIGN),
                     (dict(vh=132), ALIGN), (dict(vt=-8), ARG), (dict(dtype=7), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("inf")), ARG),
                     (dict(qw=P + 2), ALIGN), (dict(kw=P + 1), ALIGN), (dict(q=dict(x=None)), ARG), (dict(q=dict(y=P + 8)), ALIGN),
                     (dict(q=dict(heads=-1)), ARG), (dict(q=dict(heads=20000)), UNSUPPORTED), (dict(q=dict(y_head=64)), ARG),
                     (dict(q=dict(y_token=64)), ARG), (dict(q=dict(x_token=-512)), ARG),
                     (dict(total=0, start=None, k=None, pos=None, n_pos=0), OK), (dict(most=0, q="null", v=None), OK)):
        assert append(**kw) == want, (kw, orbq.load().orbq_last_error())


# ------------------------------------------------------------------------------- products with an epilogue
class Epilogue(ctypes.Structure):
    """orbq_epilogue as include/orbq.h declares it."""
    _fields_ = [("act", ctypes.c_int), ("bias", ctypes.c_void_p), ("bias_type", ctypes.c_int), ("gate", ctypes.c_void_p),
                ("gate_type", ctypes.c_int), ("gate_ld", ctypes.c_int64), ("residual", ctypes.c_void_p), ("residual_ld", ctypes.c_int64),
                ("cu", ctypes.c_void_p), ("groups", ctypes.c_int32)]


def test_the_binding_packs_the_epilogue_as_declared():
    assert orbq._EPILOGUE.size == ctypes.sizeof(Epilogue)
    values = (2, 1 << 40, 1, 3, 0, 4, 5, 6, 7, 8)
    got = Epilogue.from_buffer_copy(orbq._EPILOGUE.pack(*values))
    assert tuple(getattr(got, f[0]) for f in Epilogue._fields_) == values


EPILOGUE_ERRORS = [
    ("null", ARG), (dict(act=3), ARG), (dict(bias_type=F16), ARG), (dict(gate_type=7), ARG), (dict(groups=0), ARG), (dict(groups=3), ARG),
    (dict(gate_ld=-1), ARG), (dict(residual_ld=63), ARG), (dict(bias=P + 2), ALIGN), (dict(gate=P + 1, gate_type=BF16), ALIGN),
    (dict(cu=P + 2), ALIGN), (dict(residual=P + 2), ALIGN)]


def epilogue(e):
    f = dict(act=0, bias=P, bias_type=F32, gate=P, gate_type=F32, gate_ld=64, residual=P, residual_ld=64, cu=None, groups=2)
    f.update(e or {})
    return Epilogue(*f.values())


def test_products(cb):
    lib, d = orbq.load(), 256
    c = orbq.Codebook.from_centroids(d, 4, cb(d, 4)).struct()
    rot = orbq._Rpbh(d, 64, 0x1000, 0x2000)
    by = ctypes.byref

    def gemm(e=None, y=P, ldy=64, yt=0, n=8, x=P):
        return lib.orbq_lut_gemm_fused(x, P, by(c), P, P, by(c), n, 64, d, None if e == "null" else by(epilogue(e)), y, yt, ldy, None)

    def linear(e=None, ws_bytes=1 << 30, y=P, ldy=64, yt=0, n=8, ws=P):
        return lib.orbq_linear_fused(P, n, d, d, by(rot), by(c), 1e-8, P, P, by(c), 64, ws, ws_bytes,
                                     None if e == "null" else by(epilogue(e)), y, yt, ldy, None)

    def a16(e=None, ws_bytes=1 << 30, y=P, ldy=64, yt=0, n=8, ws=P):
        return lib.orbq_linear_a16_fused(P, n, d, d, by(rot), P, P, by(c), 64, ws, ws_bytes,
                                         None if e == "null" else by(epilogue(e)), y, yt, ldy, None)

    for f in (gemm, linear, a16):
        for e, want in EPILOGUE_ERRORS:
            assert f(e) == want, (f, e, lib.orbq_last_error())
        for kw, want in ((dict(ldy=63), ARG), (dict(yt=2), ARG), (dict(n=-1), ARG), (dict(y=None), ARG), (dict(y=P + 2), ALIGN),
                         (dict(n=0, y=None), OK)):
            assert f(**kw) == want, (f, kw, lib.orbq_last_error())
    for f in (gemm, linear):          # 16-byte pieces, 32-bit offsets within a tile
        for e, want in ((dict(residual=P + 4), ALIGN), (dict(residual_ld=66), ALIGN), (dict(residual_ld=1 << 22), UNSUPPORTED)):
            assert f(e) == want, (f, e, lib.orbq_last_error())
        assert f(ldy=1 << 22) == UNSUPPORTED
    for f in (linear, a16):
        assert f(ws_bytes=16) == WORKSPACE and f(ws=None) == WORKSPACE and f(ws=P + 16) == ALIGN
    assert gemm(x=None) == ARG


def test_the_binding_packs_rotations_and_codebooks_as_declared(cb):
    class Tensor:
        def __init__(self, at):
            self.data_ptr = lambda: at

    r = orbq._Rpbh.from_buffer_copy(orbq.Rotation(256, 64, Tensor(1 << 40), Tensor(3), 2).packed())
    assert (r.d, r.block, r.perm, r.signs, r.passes) == (256, 64, 1 << 40, 3, 2)
    assert not orbq._Rpbh.from_buffer_copy(orbq.Rotation(256, 64, None, Tensor(3)).packed()).perm
    book = orbq.Codebook.from_centroids(256, 4, cb(256, 4))
    for _ in range(2):      # the second time as kept
        c = orbq._Codebook.from_buffer_copy(book.packed())
        assert (c.d, c.bits) == (256, 4) and c.centroids[:16] == book.centroids.tolist()
    book.centroids = book.centroids * 2
    assert orbq._Codebook.from_buffer_copy(book.packed()).centroids[:16] == book.centroids.tolist()
    book.bits = 3
    assert orbq._Codebook.from_buffer_copy(book.packed()).bits == 3
    wide = orbq.Codebook(256, 4, cb(256, 4).astype("float64"))      # a copy that the codebook keeps alive
    assert orbq._Codebook.from_buffer_copy(wide.packed()).centroids[:16] == cb(256, 4).tolist()
