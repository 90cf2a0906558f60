"""CPU tests of the attention-side entry points: every argument error is caught on the host, with its
status, before anything is launched."""
import ctypes
import os

import pytest

import calibration_free_w4a4_amd as orbq

pytestmark = pytest.mark.skipif(not os.path.exists(orbq.library_path()), reason="liborbq.so not built")
P = 0x10000   # an aligned dummy device address; the host never reads it
OK, ARG, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4


class Structs:
    """The C structs as include/orbq.h declares them."""
    class _Rope(ctypes.Structure):
        _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * 4), ("freqs", ctypes.c_void_p), ("layout", ctypes.c_int)]

    class _Heads(ctypes.Structure):
        _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int32)] + \
            [(n, ctypes.c_int64) for n in ("x_token", "x_head", "y_token", "y_head")]

    class _Cache(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + \
            [(n, ctypes.c_int32) for n in ("num_pages", "kv_heads", "page_tokens", "head_dim")]

    class _Table(ctypes.Structure):
        _fields_ = [("table", ctypes.c_void_p), ("ld", ctypes.c_int64), ("max_pages", ctypes.c_int32), ("batch", ctypes.c_int32)]


def structs():
    return Structs


def test_the_binding_packs_the_structs_as_declared():
    from calibration_free_w4a4_amd import attention as at
    for mine, theirs in ((at._ROPE, Structs._Rope), (at._HEADS, Structs._Heads), (at._CACHE, Structs._Cache),
                         (at._TABLE, Structs._Table)):
        assert mine.size == ctypes.sizeof(theirs)
    r = Structs._Rope.from_buffer_copy(at._ROPE.pack(3, 44, 42, 40, 2, 1 << 40, 1))
    assert (r.axes, list(r.dims), r.freqs, r.layout) == (3, [44, 42, 40, 2], 1 << 40, 1)
    h = Structs._Heads.from_buffer_copy(at._HEADS.pack(1, 2, 3, -4, 5, 6, 7))
    assert (h.x, h.y, h.heads, h.x_token, h.x_head, h.y_token, h.y_head) == (1, 2, 3, -4, 5, 6, 7)
    c = Structs._Cache.from_buffer_copy(at._CACHE.pack(1, 2, 3, 4, 5, 6, 7, 8))
    assert [getattr(c, f[0]) for f in c._fields_] == [1, 2, 3, 4, 5, 6, 7, 8]
    t = Structs._Table.from_buffer_copy(at._TABLE.pack(1, 2, 3, 4))
    assert [getattr(t, f[0]) for f in t._fields_] == [1, 2, 3, 4]


def rope_call(dims=(44, 42, 42), axes=None, freqs=P, layout=0, pos=P, n_pos=8, n=8, d=128, x=P, y=P, heads=2, strides=None,
              count=1, dtype=1, null=None):
    at = structs()
    r = at._Rope(len(dims) if axes is None else axes, (ctypes.c_int32 * 4)(*dims[:4]), freqs, layout)
    t = (at._Heads * 2)()
    for i in range(2):
        t[i] = at._Heads(x, y, heads, *(strides or (heads * d, d, heads * d, d)))
    return orbq.load().orbq_rope_apply(None if null == "rope" else ctypes.byref(r), pos, n_pos, n, d,
                                       None if null == "tensors" else t, count, dtype, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(null="rope"), ARG), (dict(null="tensors"), ARG), (dict(axes=0), UNSUPPORTED), (dict(axes=5), UNSUPPORTED),
    (dict(dims=(43, 42, 42)), ARG), (dict(dims=(-2, 42)), ARG), (dict(dims=(64, 66)), ARG), (dict(dims=(0, 0)), ARG),
    (dict(d=127, dims=(2,)), UNSUPPORTED), (dict(d=514, dims=(2,)), UNSUPPORTED), (dict(layout=2), ARG), (dict(dtype=3), ARG),
    (dict(n=-1), ARG), (dict(count=0), ARG), (dict(count=3), ARG), (dict(n_pos=0), ARG), (dict(n_pos=3), ARG),
    (dict(pos=None), ARG), (dict(freqs=None), ARG), (dict(pos=P + 2), ALIGN), (dict(x=None), ARG), (dict(y=None), ARG),
    (dict(heads=-1), ARG), (dict(strides=(-1, 128, 256, 128)), ARG), (dict(strides=(256, 128, 256, 64)), ARG),
    (dict(strides=(256, 128, 64, 128)), ARG), (dict(x=P + 1), ALIGN), (dict(x=P + 2, dtype=0), ALIGN),
    (dict(n=1 << 31, n_pos=1), UNSUPPORTED), (dict(heads=20000), UNSUPPORTED),
    (dict(n=0, pos=None, x=None, y=None, freqs=None), OK), (dict(heads=0, x=None, y=None), OK)])
def test_rope(kw, want):
    assert rope_call(**kw) == want, orbq.load().orbq_last_error().decode()


def cache(at, **kw):
    f = dict(k_codes=P, v_codes=P, k_scales=P, v_scales=P, num_pages=8, kv_heads=2, page_tokens=64, head_dim=128)
    f.update(kw)
    return at._Cache(**f)


CACHE_ERRORS = [
    (dict(head_dim=96), {}, UNSUPPORTED), (dict(page_tokens=48), {}, UNSUPPORTED), (dict(num_pages=0), {}, ARG),
    (dict(kv_heads=0), {}, ARG), (dict(kv_heads=20000), {}, UNSUPPORTED), (dict(k_codes=None), {}, ARG), (dict(v_scales=None), {}, ARG),
    (dict(k_codes=P + 8), {}, ALIGN), (dict(v_codes=P + 8), {}, ALIGN), (dict(k_scales=P + 2), {}, ALIGN), ({}, dict(table=None), ARG),
    ({}, dict(batch=-1), ARG), ({}, dict(ld=3), ARG), ({}, dict(max_pages=-1), ARG), ({}, dict(batch=70000), UNSUPPORTED),
    ({}, dict(max_pages=1 << 25, ld=1 << 25), UNSUPPORTED), ({}, dict(table=P + 2), ALIGN)]


def table(at, **kw):
    f = dict(table=P, ld=4, max_pages=4, batch=2)
    f.update(kw)
    return at._Table(**f)


def move(read, c=None, t=None, first=P, cu=P, total=6, most=3, k=P, kt=256, kh=128, v=P, vt=256, vh=128, dtype=1):
    at = structs()
    lib = orbq.load()
    f = lib.orbq_kv_read if read else lib.orbq_kv_append
    c = None if c == "null" else ctypes.byref(cache(at, **(c or {})))
    t = None if t == "null" else ctypes.byref(table(at, **(t or {})))
    return f(c, t, first, cu, total, most, k, kt, kh, v, vt, vh, dtype, None)


@pytest.mark.parametrize("read", [False, True])
def test_append_and_read(read):
    for c, t, want in CACHE_ERRORS:
        assert move(read, c, t) == want, (c, t, orbq.load().orbq_last_error())
    for kw, want in ((dict(c="null"), ARG), (dict(t="null"), ARG), (dict(first=None), ARG), (dict(first=P + 1), ALIGN),
                     (dict(cu=P + 2), ALIGN), (dict(cu=None, total=5), ARG), (dict(total=-1), ARG), (dict(most=-1), ARG),
                     (dict(t=dict(batch=0)), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=P + 8), ALIGN),
                     (dict(kt=260), ALIGN), (dict(vh=132), ALIGN), (dict(kt=-256), ARG), (dict(dtype=4), ARG),
                     (dict(total=1 << 31), UNSUPPORTED), (dict(total=0, first=None, k=None), OK), (dict(most=0, v=None), OK)):
        assert move(read, **kw) == want, (kw, orbq.load().orbq_last_error())
    if read:        # rows that would overlap
        assert move(True, kt=64) == ARG and move(True, vh=64) == ARG


def attend(c=None, t=None, lens=P, cu=P, total=6, most=3, max_len=0, q=P, qt=512, qh=128, heads=4, o=P, ot=512, oh=128,
           lse=None, dtype=1, scale=0.1, block=0, window=0, ws=None, ws_bytes=0):
    at = structs()
    c = None if c == "null" else ctypes.byref(cache(at, **(c or {})))
    t = None if t == "null" else ctypes.byref(table(at, **(t or {})))
    return orbq.load().orbq_kv_attention(c, t, lens, cu, total, most, max_len, q, qt, qh, heads, o, ot, oh, lse, dtype, scale,
                                         block, window, ws, ws_bytes, None)


def test_attention():
    for c, t, want in CACHE_ERRORS:
        assert attend(c, t) == want, (c, t, orbq.load().orbq_last_error())
    long = dict(max_pages=8000, ld=8000)
    for kw, want in ((dict(c="null"), ARG), (dict(t="null"), ARG), (dict(lens=None), ARG), (dict(lens=P + 2), ALIGN),
                     (dict(heads=3), ARG), (dict(heads=0), ARG), (dict(heads=20000), UNSUPPORTED), (dict(max_len=-1), ARG),
                     (dict(block=-1), ARG), (dict(window=-1), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
                     (dict(dtype=0), UNSUPPORTED), (dict(dtype=5), ARG), (dict(q=None), ARG), (dict(o=None), ARG),
                     (dict(q=P + 8), ALIGN), (dict(qh=132), ALIGN), (dict(o=P + 4), ALIGN), (dict(ot=510), ALIGN),
                     (dict(ot=64), ARG), (dict(oh=64), ARG), (dict(lse=P + 2), ALIGN), (dict(cu=None, total=5), ARG),
                     (dict(most=1 << 30, heads=256), UNSUPPORTED), (dict(t=long), WORKSPACE), (dict(t=long, ws=P, ws_bytes=100), WORKSPACE),
                     (dict(t=long, ws=P + 16, ws_bytes=1 << 40), ALIGN),
                     (dict(total=0, q=None, o=None, lens=None), OK), (dict(most=0, q=None), OK)):
        assert attend(**kw) == want, (kw, orbq.load().orbq_last_error())


def test_workspace_bytes():
    at = structs()
    lib = orbq.load()
    f = lambda *a: lib.orbq_kv_attention_workspace_bytes(ctypes.byref(cache(at)), *a)  # noqa: E731
    assert f(48, 48, 1, 8, 64, 0, 0) == 0                     # one 64-key tile is not split
    n = f(1, 1, 1, 2, 200000, 0, 0)
    assert n > 0 and n % ((128 + 2) * 4) == 0                  # parts of 2 rows: d values, m and l each
    assert f(1, 1, 1, 2, 200000, 1, 64) < n                     # a window leaves little to split
    assert f(0, 1, 1, 2, 64, 0, 0) == 0 and f(1, 1, 1, 3, 10 ** 6, 0, 0) == 0 and f(1, 1, 1, 2, -1, 0, 0) == 0
    assert lib.orbq_kv_attention_workspace_bytes(None, 1, 1, 1, 2, 64, 0, 0) == 0
