"""Binding of the attention-side operators: rotary positions with several axes, the 8-bit paged
key/value cache, attention over it (include/orbq.h says what each computes).  As elsewhere in this
package the functions only check and marshal arguments; the work is liborbq's HIP kernels.

    r = Rope.create((44, 42, 42))                          # entries a head turns by time, height, width
    q, k = rope(r, positions, q, k)                        # gradients: rope_backward(r, positions, dq, dk)
    cache = KVCache.create(num_pages, kv_heads, head_dim)  # int8 codes, a scale for each page and head
    kv_append(cache, k, v, table, held)                    # quantise and write behind `held` tokens
    o = kv_attention(cache, q, table, lens, causal_block=tokens_a_frame)

Head tensors are [tokens, heads, head_dim] with the last dimension contiguous.

Gradients: rope and rope_backward are part of the autograd graph (positions and frequencies are constants).  There is no
gradient through the cache, whose entries are rounded: a backward pass that reaches kv_attention's output raises.  A call
that is given `out` writes it and records nothing.
"""
from __future__ import annotations

import functools
import operator
import struct

from . import OrbqError, _check, load

__all__ = ["Rope", "rope", "rope_backward", "KVCache", "kv_append", "kv_read", "kv_attention",
           "kv_attention_workspace_bytes"]

# torch comes with the first Rope or KVCache, which every call takes: the package can be imported, with all its names,
# where there is none.
torch = None
_TYPES = {}
_Turned = _Attended = None  # autograd functions of rope and kv_attention


def _need_torch() -> None:
    global torch, _Turned, _Attended
    if torch is not None:
        return
    import torch as t

    class Turned(t.autograd.Function):
        """The map is linear and orthogonal: its gradient is the inverse turn, whose gradient is the turn again."""
        @staticmethod
        def forward(ctx, func, rope, positions, q, k, inverse):
            ctx.func, ctx.rope, ctx.inverse = func, rope, inverse
            ctx.save_for_backward(positions)
            ctx.set_materialize_grads(False)
            return _turn(func, rope, positions, q, k, inverse, None)

        @staticmethod
        def backward(ctx, *dy):
            positions, = ctx.saved_tensors
            # the gradients that are there and asked for, in one launch; an expanded one has no contiguous last dimension
            some = [i for i, g in enumerate(dy) if g is not None and ctx.needs_input_grad[3 + i]]
            dx = [None, None]
            if some:
                dy = [dy[i] if dy[i].stride(-1) == 1 else dy[i].contiguous() for i in some]
                got = _turn(ctx.func, ctx.rope, positions, dy[0], dy[1] if len(dy) > 1 else None, 1 - ctx.inverse, None)
                for i, g in zip(some, got if len(some) > 1 else (got,)):
                    dx[i] = g
            return None, None, None, *dx, None

    class Attended(t.autograd.Function):
        @staticmethod
        def forward(ctx, cache, q, *args):
            return kv_attention(cache, q, *args)

        @staticmethod
        def backward(ctx, do):
            raise _bad("kv_attention", "there is no gradient through the 8-bit cache")

    _TYPES.update({t.float32: 0, t.bfloat16: 1, t.float16: 2})
    _Turned, _Attended = Turned, Attended
    torch = t


LAYOUTS = {"pairs": 0, "halves": 1}  # orbq_rope_layout

# The C structs, packed (a token step's calls are short: building ctypes structures would cost as much as
# the kernels take to start).
_ROPE = struct.Struct("<5i4xQi4x")       # orbq_rope
_HEADS = struct.Struct("<QQi4x4q")       # orbq_heads
_CACHE = struct.Struct("<4Q4i")          # orbq_kv_cache
_TABLE = struct.Struct("<Qqii")          # orbq_page_table


def _bad(func: str, detail: str) -> OrbqError:
    return OrbqError(-1, func, detail)


def _stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)  # torch.cuda.current_stream(device).cuda_stream, 2 us less


def _current() -> int:
    """The current device.  A stream's raw handle (0 for every device's default one) means a stream of that device, so each
    call below makes the tensors' device current first."""
    return torch._C._cuda_getDevice()


def _lay(t, func: str, name: str):
    """(tokens, heads, head_dim, token stride, head stride, address, type) of a head tensor: on the GPU, [tokens,
    heads, head_dim] with contiguous heads.  A dimension of one entry has no stride of its own: 0."""
    if t.dim() != 3:
        raise _bad(func, f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    a, b, c = t.stride()
    if c != 1 and d > 1:
        raise _bad(func, f"{name} must have a contiguous last dimension")
    code = _TYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        raise _bad(func, f"{name} must be float32, bfloat16 or float16 on the GPU, got {t.dtype} on {t.device}")
    return n, h, d, a if n > 1 else 0, b if h > 1 else 0, t.data_ptr(), code


def _ints(t, device: int, count: int, func: str, name: str) -> int:
    if t.dtype != torch.int32 or t.get_device() != device or t.shape != (count,) or not t.is_contiguous():
        raise _bad(func, f"{name} must be contiguous int32 [{count}] on cuda:{device}")
    return t.data_ptr()


def _fixed(cls):
    """Gives the private slots of `cls` public names that cannot be set: the packed C struct holds their values and
    addresses, and would go on holding those of a tensor that is gone."""
    for name in cls.__slots__:
        setattr(cls, name[1:], property(operator.attrgetter(name)))
    return cls


# ------------------------------------------------------------------------------------ rotary positions
@_fixed
class Rope:
    """dims: entries of a head that each axis turns (even; in order from entry 0; the rest of the head
    passes through).  freqs: float32 [sum(dims) / 2] on the GPU, radians per unit of position for each
    pair.  layout: "pairs" (2 i, 2 i + 1) or "halves" (i, i + sum(dims) / 2).  Attributes are read only."""
    __slots__ = ("_dims", "_freqs", "_layout", "_packed", "_device")

    def __init__(self, dims, freqs, layout: str = "pairs"):
        _need_torch()
        dims = tuple(dims)
        if not 1 <= len(dims) <= 4 or layout not in LAYOUTS:
            raise _bad("Rope", f"{len(dims)} axes (1 to 4), layout {layout!r} (one of {sorted(LAYOUTS)})")
        if freqs.dtype != torch.float32 or not freqs.is_cuda or freqs.shape != (sum(dims) // 2,) or not freqs.is_contiguous():
            raise _bad("Rope", f"freqs must be contiguous float32 [{sum(dims) // 2}] on the GPU")
        self._dims, self._freqs, self._layout, self._device = dims, freqs, layout, freqs.get_device()
        self._packed = _ROPE.pack(len(dims), *dims, *(0,) * (4 - len(dims)), freqs.data_ptr(), LAYOUTS[layout])

    @classmethod
    def create(cls, dims, theta: float = 10000.0, layout: str = "pairs", device=None) -> "Rope":
        """Frequencies theta^(-2 i / dims[a]) for pair i of axis a."""
        _need_torch()
        f = torch.cat([theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims])
        return cls(tuple(dims), f.float().to(device or torch.device("cuda", torch.cuda.current_device())), layout)


def _like(x):
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _written(x, y, func: str):
    """Token and head strides of the output y given for x."""
    if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device:
        raise _bad(func, "out must have the inputs' shapes, types and device")
    return _lay(y, func, "out")[3:5]


def _turn(func, rope, positions, q, k, inverse, out):
    if out is None and (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        return _Turned.apply(func, rope, positions, q, k, inverse)      # which comes back here, recording nothing
    if _current() != rope._device:
        with torch.cuda.device(rope._device):
            return _turn(func, rope, positions, q, k, inverse, out)
    n, h, d, xt, xh, x, code = _lay(q, func, "q")
    dev = rope._device
    if q.get_device() != dev:
        raise _bad(func, f"q must be on cuda:{dev}, where the frequencies are")
    if positions.dtype != torch.float32 or positions.get_device() != dev or positions.dim() != 2 or \
            positions.shape[1] != len(rope._dims) or not positions.is_contiguous():
        raise _bad(func, f"positions must be contiguous float32 [tokens, {len(rope._dims)}] on cuda:{dev}")
    if out is not None:
        yq, yk = (out, None) if k is None else out
    else:
        yq = _like(q)
    heads = _HEADS.pack(x, yq.data_ptr(), h, xt, xh, *((h * d, d) if out is None else _written(q, yq, func)))
    if k is not None:
        n2, h, d2, xt, xh, x, code2 = _lay(k, func, "k")
        if n2 != n or d2 != d or code2 != code or k.get_device() != dev:
            raise _bad(func, "q and k must agree in tokens, head_dim, type and device")
        if out is None:
            yk = _like(k)
        heads += _HEADS.pack(x, yk.data_ptr(), h, xt, xh, *((h * d, d) if out is None else _written(k, yk, func)))
    st = load().orbq_rope_apply(rope._packed, positions.data_ptr(), positions.shape[0], n, d, heads, 1 if k is None else 2,
                                code, inverse, _stream(dev))
    if st:
        _check(st, "orbq_rope_apply")
    return yq if k is None else (yq, yk)


def rope(rope: Rope, positions, q, k=None, out=None):
    """q (and k, in the same launch) [tokens, heads, head_dim] turned by their positions float32
    [tokens or a divisor of it, axes].  out: where to write, one tensor for each input (the inputs
    themselves: in place)."""
    return _turn("rope", rope, positions, q, k, 0, out)


def rope_backward(rope: Rope, positions, dq, dk=None, out=None):
    """Gradients of rope's inputs from those of its outputs (the transposed map)."""
    return _turn("rope_backward", rope, positions, dq, dk, 1, out)


# ------------------------------------------------------------------------------------------ the cache
@_fixed
class KVCache:
    """k_codes int8 [pages, kv_heads, page_tokens, head_dim], v_codes int8 [pages, kv_heads, head_dim,
    page_tokens], k_scales and v_scales float32 [pages, kv_heads], all contiguous on one GPU.  Attributes are read
    only; what the tensors hold may be written."""
    __slots__ = ("_k_codes", "_v_codes", "_k_scales", "_v_scales", "_kv_heads", "_page_tokens", "_head_dim", "_packed", "_device")

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        _need_torch()
        if k_codes.dim() != 4:
            raise _bad("KVCache", "k_codes must be [pages, kv_heads, page_tokens, head_dim]")
        n, h, t, d = k_codes.shape
        dev = k_codes.get_device()
        for x, shape, kind in ((k_codes, (n, h, t, d), torch.int8), (v_codes, (n, h, d, t), torch.int8),
                               (k_scales, (n, h), torch.float32), (v_scales, (n, h), torch.float32)):
            if x.shape != shape or x.dtype != kind or x.get_device() != dev or dev < 0 or not x.is_contiguous():
                raise _bad("KVCache", f"expected contiguous {kind} {shape} on one GPU, got {x.dtype} {tuple(x.shape)} on {x.device}")
        self._k_codes, self._v_codes, self._k_scales, self._v_scales = k_codes, v_codes, k_scales, v_scales
        self._kv_heads, self._page_tokens, self._head_dim, self._device = h, t, d, dev
        self._packed = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), n, h, t, d)

    @classmethod
    def create(cls, num_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device=None) -> "KVCache":
        _need_torch()
        dev = device or torch.device("cuda", torch.cuda.current_device())
        code = lambda *s: torch.empty(s, dtype=torch.int8, device=dev)  # noqa: E731
        scale = lambda: torch.empty((num_pages, kv_heads), dtype=torch.float32, device=dev)  # noqa: E731
        return cls(code(num_pages, kv_heads, page_tokens, head_dim), code(num_pages, kv_heads, head_dim, page_tokens),
                   scale(), scale())


def _table(table, cache, func: str):
    """(packed page table, batch, pages a row)"""
    if table.dtype != torch.int32 or table.get_device() != cache._device or table.dim() != 2:
        raise _bad(func, f"table must be int32 [batch, pages] on cuda:{cache._device}")
    b, p = table.shape
    ld, one = table.stride()
    if one != 1 and p > 1:
        raise _bad(func, "table must have contiguous rows")
    return _TABLE.pack(table.data_ptr(), ld if b > 1 else p, p, b), b, p


def _move(func, entry, cache, k, v, table, first, cu, most):
    if _current() != cache._device:
        with torch.cuda.device(cache._device):
            return _move(func, entry, cache, k, v, table, first, cu, most)
    t, batch, _ = _table(table, cache, func)
    n, h, d, kt, kh, kp, code = _lay(k, func, "k")
    nv, hv, dv, vt, vh, vp, code_v = _lay(v, func, "v")
    dev = cache._device
    if h != cache._kv_heads or d != cache._head_dim or (nv, hv, dv, code_v) != (n, h, d, code) or k.get_device() != dev or \
            v.get_device() != dev:
        raise _bad(func, f"k and v must be [tokens, {cache._kv_heads}, {cache._head_dim}] of one type on cuda:{dev}")
    first = _ints(first, dev, batch, func, "positions")
    cu = 0 if cu is None else _ints(cu, dev, batch + 1, func, "cu")
    if most is None:
        most = n if cu else n // max(1, batch)
    st = entry(cache._packed, t, first, cu, n, most, kp, kt, kh, vp, vt, vh, code, _stream(dev))
    if st:
        _check(st, "orbq_" + func)


def kv_append(cache: KVCache, k, v, table, start, cu=None, max_new=None) -> None:
    """Quantises k, v [total, kv_heads, head_dim] and writes them behind the start[b] tokens that sequence b
    holds.  table int32 [batch, pages]; start int32 [batch]; cu int32 [batch + 1]: rows of each sequence (None:
    equal shares); max_new: no sequence has more (None: the most there can be)."""
    _move("kv_append", load().orbq_kv_append, cache, k, v, table, start, cu, max_new)


def kv_read(cache: KVCache, table, first, cu, total: int, max_tokens=None, dtype=None, out=None):
    """(k, v) [total, kv_heads, head_dim] of tokens first[b] .. of each sequence, cu as in kv_append.  dtype: of the
    result (None: torch.bfloat16)."""
    if out is None:
        dtype = dtype or torch.bfloat16
        k = cache._k_scales.new_empty((total, cache._kv_heads, cache._head_dim), dtype=dtype)
        out = (k, torch.empty_like(k))
    elif out[0].shape[0] != total:
        raise _bad("kv_read", f"out must have {total} tokens")
    _move("kv_read", load().orbq_kv_read, cache, out[0], out[1], table, first, cu, max_tokens)
    return out


# ---------------------------------------------------------------------------------------- attention
def kv_attention_workspace_bytes(cache: KVCache, batch: int, total: int, max_new: int, heads: int, max_len: int,
                                 causal_block: int = 0, window: int = 0) -> int:
    with torch.cuda.device(cache._device):
        return int(load().orbq_kv_attention_workspace_bytes(cache._packed, batch, total, max_new, heads, max_len, causal_block,
                                                            window))


@functools.lru_cache(maxsize=1024)
def _workspace(kv_heads, head_dim, device, *sizes) -> int:
    # the plan goes by these sizes alone (and the device's compute units)
    return int(load().orbq_kv_attention_workspace_bytes(_CACHE.pack(0, 0, 0, 0, 1, kv_heads, 16, head_dim), *sizes))


def kv_attention(cache: KVCache, q, table, lens, cu=None, max_new=None, causal_block: int = 0, window: int = 0,
                 scale=None, max_len=None, out=None, lse=None, workspace=None):
    """Attention of packed queries q [total, heads, head_dim] (bf16 or f16) over the cache; query i of the n of
    sequence b stands at position lens[b] - n + i.  causal_block: 0 none, 1 causal, tokens a frame: each frame
    sees itself and earlier ones.  window: at most that many of the latest visible tokens (0: all).  scale:
    1 / sqrt(head_dim) if None.  lse: float32 [total, heads] to receive the logarithms of the sums.
    max_len: expected bound of lens (None or 0: what the table holds); it only guides how the work is split."""
    func = "kv_attention"
    if q.requires_grad and out is None and torch.is_grad_enabled():
        return _Attended.apply(cache, q, table, lens, cu, max_new, causal_block, window, scale, max_len, out, lse, workspace)
    if _current() != cache._device:
        with torch.cuda.device(cache._device):
            return kv_attention(cache, q, table, lens, cu, max_new, causal_block, window, scale, max_len, out, lse, workspace)
    t, batch, pages = _table(table, cache, func)
    n, h, d, qt, qh, qp, code = _lay(q, func, "q")
    dev = cache._device
    if d != cache._head_dim or q.get_device() != dev:
        raise _bad(func, f"q must be [tokens, heads, {cache._head_dim}] on cuda:{dev}")
    lens = _ints(lens, dev, batch, func, "lens")
    cu = 0 if cu is None else _ints(cu, dev, batch + 1, func, "cu")
    if max_new is None:
        max_new = n if cu else n // max(1, batch)
    if out is None:
        out, ot, oh = _like(q), h * d, d
    else:
        ot, oh = _written(q, out, func)
    if lse is not None and (lse.shape != (n, h) or lse.dtype != torch.float32 or lse.get_device() != dev or
                            not lse.is_contiguous()):
        raise _bad(func, f"lse must be contiguous float32 [{n}, {h}] on cuda:{dev}")
    held = pages * cache._page_tokens
    max_len = held if not max_len or max_len > held else max_len
    lib = load()
    if workspace is None:
        need = _workspace(cache._kv_heads, d, dev, batch, n, max_new, h, max_len, causal_block, window)
        if need:
            workspace = q.new_empty((need + 1) // 2)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise _bad(func, f"workspace must be contiguous on cuda:{dev}")
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = lib.orbq_kv_attention(cache._packed, t, lens, cu, n, max_new, max_len, qp, qt, qh, h, out.data_ptr(), ot, oh,
                               0 if lse is None else lse.data_ptr(), code, d ** -0.5 if scale is None else scale, causal_block,
                               window, ws, ws_bytes, _stream(dev))
    if st:
        _check(st, "orbq_kv_attention")
    return out
