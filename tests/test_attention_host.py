"""CPU tests of the attention-side host layer: what it makes of bounds, strides, devices and attributes."""
import ctypes
import os

import pytest

import calibration_free_w4a4_amd as orbq
from tests.test_attention_abi import Structs, cache

pytestmark = pytest.mark.skipif(not os.path.exists(orbq.library_path()), reason="liborbq.so not built")


@pytest.mark.parametrize("batch,total,max_len,d", [(1, 1, 200000, 128), (48, 48, 16384, 128), (1, 4, 262144, 64), (3, 700, 5000, 256)])
def test_a_bound_above_the_work_changes_no_plan(batch, total, max_len, d):
    """One bound for every call of a loop: max_new far above `total` plans as `total` does."""
    c = cache(Structs, head_dim=d)
    size = lambda most: orbq.load().orbq_kv_attention_workspace_bytes(ctypes.byref(c), batch, total, most, 8, max_len, 1, 0)  # noqa: E731
    assert size(total) > 0
    for most in (total + 1, 1000 * total, 2 ** 30):
        assert size(most) == size(total)


class Elsewhere:
    """A CPU tensor that says it is on cuda:1."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def two_devices(monkeypatch):
    """cuda:0 is current; the library's entry points note which device is when they are called."""
    torch = pytest.importorskip("torch")
    from calibration_free_w4a4_amd import attention as at
    current, seen = [0], []

    class on:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *args):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                seen.append((name, current[0]))
                return 0
            return entry

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", on)
    for m in (orbq, at):
        monkeypatch.setattr(m, "load", lambda: Library())
    monkeypatch.setattr(at, "_stream", lambda device: 0)
    monkeypatch.setattr(orbq, "_stream", lambda torch, device: 0)
    monkeypatch.setattr(orbq, "_torch", lambda: torch)
    at._workspace.cache_clear()
    yield seen
    at._workspace.cache_clear()
    assert current[0] == 0


def launches(seen):
    sizes = ("workspace_bytes", "row_bytes")      # the second goes by no device
    return [(n, d) for n, d in seen if not n.endswith(sizes[1])]


def test_attention_calls_run_on_the_tensors_device(two_devices):
    import torch
    from calibration_free_w4a4_amd import attention as at
    x = lambda *s, dtype=torch.bfloat16: Elsewhere(torch.zeros(s, dtype=dtype))  # noqa: E731
    r = at.Rope((32,), x(16, dtype=torch.float32))
    q, pos = x(4, 2, 64), x(4, 1, dtype=torch.float32)
    at.rope(r, pos, q, out=x(4, 2, 64))
    at.rope_backward(r, pos, q, q, out=(x(4, 2, 64), x(4, 2, 64)))
    c = at.KVCache(x(3, 2, 16, 64, dtype=torch.int8), x(3, 2, 64, 16, dtype=torch.int8), x(3, 2, dtype=torch.float32),
                   x(3, 2, dtype=torch.float32))
    table, lens = x(1, 3, dtype=torch.int32), x(1, dtype=torch.int32)
    at.kv_append(c, q, q, table, lens)
    at.kv_read(c, table, lens, None, 4, out=(x(4, 2, 64), x(4, 2, 64)))
    at.kv_attention(c, q, table, lens, out=x(4, 2, 64))
    at.kv_attention_workspace_bytes(c, 1, 4, 4, 2, 48)
    assert [n for n, _ in two_devices] == ["orbq_rope_apply"] * 2 + ["orbq_kv_append", "orbq_kv_read"] + \
        ["orbq_kv_attention_workspace_bytes", "orbq_kv_attention", "orbq_kv_attention_workspace_bytes"]
    assert all(device == 1 for _, device in two_devices)


def test_layer_calls_run_on_the_tensors_device(two_devices):
    import numpy as np
    import torch
    x = lambda *s, dtype=torch.bfloat16: Elsewhere(torch.zeros(s, dtype=dtype))  # noqa: E731
    rot = orbq.Rotation(64, 64, None, torch.zeros(64, dtype=torch.int8))
    cb = orbq.Codebook.from_centroids(64, 4, np.arange(16) - 7.5)
    X, codes, norms, y = x(2, 64), x(2, 32, dtype=torch.uint8), x(2, dtype=torch.float32), x(2, 2, dtype=torch.float32)
    both = dict(out_codes=codes, out_norms=norms)
    orbq.fold_weights(X, rot, cb, **both)
    orbq.rpbh_quantize(X=X, rot=rot, cb=cb, **both)
    orbq.lut_gemm(codes, norms, cb, codes, norms, cb, 64, out=y)
    orbq.linear(X, rot, cb, codes, norms, cb, workspace=x(512, dtype=torch.uint8), out=y)
    orbq.linear_noalloc(X, rot, cb, codes, norms, cb, out=y)
    orbq.linear_a16(X, rot, codes, norms, cb, workspace=x(512, dtype=torch.uint8), out=y)
    orbq.flatness(X)
    orbq.test_rotate(X, rot)
    orbq.test_quantize_t(norms, cb)
    got = launches(two_devices)
    assert len(got) == 11 and all(device == 1 for _, device in got), got      # nine launches, two sizes


def test_what_the_packed_structs_hold_cannot_be_replaced():
    """The C structs keep the tensors' addresses: a tensor set on the object would not be used, and the one that it
    replaced might be freed."""
    torch = pytest.importorskip("torch")
    from calibration_free_w4a4_amd import attention as at
    x = lambda *s, dtype: Elsewhere(torch.zeros(s, dtype=dtype))  # noqa: E731
    freqs = x(16, dtype=torch.float32)
    r = at.Rope((32,), freqs, "halves")
    assert (r.dims, r.layout, r.device) == ((32,), "halves", 1) and r.freqs is freqs
    codes, scales = x(3, 2, 16, 64, dtype=torch.int8), x(3, 2, dtype=torch.float32)
    c = at.KVCache(codes, x(3, 2, 64, 16, dtype=torch.int8), scales, scales)
    assert c.k_codes is codes and c.v_scales is scales and (c.kv_heads, c.page_tokens, c.head_dim, c.device) == (2, 16, 64, 1)
    for o, names in ((r, "dims freqs layout packed device"),
                     (c, "k_codes v_codes k_scales v_scales kv_heads page_tokens head_dim packed device")):
        for name in names.split():
            with pytest.raises(AttributeError):
                setattr(o, name, getattr(o, name))


@pytest.mark.parametrize("tokens,heads,width", [(6, 4, 64), (2, 2, 64), (5, 7, 64), (1, 4, 64), (9, 1, 64)])
def test_outputs_whose_rows_overlap_are_refused(tokens, heads, width):
    """Against all pairs of rows, for strides around the row's width and in both orders of tokens and heads."""
    import itertools
    P, lib = 0x10000, orbq.load()
    r = Structs._Rope(1, (ctypes.c_int32 * 4)(width), P, 0)
    steps = sorted({width // 2, width - 2, width, width + 2, 2 * width, 3 * width, 3 * width + 2, heads * width - 2, heads * width,
                    tokens * width - 2, tokens * width, tokens * width + 6, 5 * width // 2})
    some = [0, 0]
    for ts, hs in itertools.product(steps, steps):
        rows = sorted(i * ts + j * hs for i in range(tokens) for j in range(heads))
        bad = any(b - a < width for a, b in zip(rows, rows[1:]))
        # the second tensor is refused in any case, with another status, so that nothing is launched
        t = (Structs._Heads * 2)(Structs._Heads(P, P, heads, heads * width, width, ts, hs),
                                 Structs._Heads(P, P, 20000, 128, 64, 128, 64))
        status = lib.orbq_rope_apply(ctypes.byref(r), P, tokens, tokens, width, t, 2, 1, 0, None)
        assert status == (-1 if bad else -2), (ts, hs, status, lib.orbq_last_error())
        some[bad] += 1
    assert all(some)


def test_the_package_is_imported_without_torch():
    """All its names, as before there were any that work on tensors alone."""
    import subprocess
    import sys
    code = ("import sys\nsys.modules['torch'] = None\nfrom calibration_free_w4a4_amd import *\n"
            "assert callable(rope) and callable(kv_attention) and KVCache and Codebook\n"
            "assert Codebook.lloyd_max(64, 4).centroids.shape == (16,)")
    root = os.path.dirname(os.path.dirname(os.path.abspath(orbq.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_products_refuse_outputs_of_other_types(two_devices):
    """Narrower ones would be written beyond their end."""
    import numpy as np
    import torch
    x = lambda *s, dtype=torch.bfloat16: Elsewhere(torch.zeros(s, dtype=dtype))  # noqa: E731
    rot = orbq.Rotation(64, 64, None, torch.zeros(64, dtype=torch.int8))
    cb = orbq.Codebook.from_centroids(64, 4, np.arange(16) - 7.5)
    X, codes, norms, ws = x(2, 64), x(2, 32, dtype=torch.uint8), x(2, dtype=torch.float32), x(512, dtype=torch.uint8)
    calls = [lambda **kw: orbq.lut_gemm(codes, norms, cb, codes, norms, cb, 64, **kw),
             lambda **kw: orbq.linear(X, rot, cb, codes, norms, cb, workspace=ws, **kw),
             lambda **kw: orbq.linear_noalloc(X, rot, cb, codes, norms, cb, **kw),
             lambda **kw: orbq.linear_a16(X, rot, codes, norms, cb, workspace=ws, **kw)]
    for call in calls:
        for kw in (dict(out_dtype=torch.float16), dict(out=x(2, 2, dtype=torch.float16)), dict(out=x(2, 2, dtype=torch.int8))):
            with pytest.raises(orbq.OrbqError):
                call(**kw)
        for dt in (torch.float32, torch.bfloat16):
            assert call(out_dtype=dt).dtype == dt
    assert not [n for n, _ in two_devices if not n.endswith("bytes")][8:]
