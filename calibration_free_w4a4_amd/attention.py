"""Binding of the attention-side operators: rotary positions with several axes, the 8-bit paged
key/value cache, attention over it (include/orbq.h says what each computes).  As elsewhere in this
package the functions only check and marshal arguments; the work is liborbq's HIP kernels.

    r = Rope.create((44, 42, 42))                          # entries a head turns by time, height, width
    q, k = rope(r, positions, q, k)                        # gradients: rope_backward(r, positions, dq, dk)
    cache = KVCache.create(num_pages, kv_heads, head_dim)  # int8 codes, a scale for each page and head
    kv_append(cache, k, v, table, held)                    # quantise and write behind `held` tokens
    o = kv_attention(cache, q, table, lens, causal_block=tokens_a_frame)

Head tensors are [tokens, heads, head_dim] with the last dimension contiguous.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import OrbqError, _check, load

__all__ = ["Rope", "rope", "rope_backward", "KVCache", "kv_append", "kv_read", "kv_attention",
           "kv_attention_workspace_bytes"]

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
LAYOUTS = {"pairs": 0, "halves": 1}  # orbq_rope_layout


class _Rope(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * 4), ("freqs", ctypes.c_void_p),
                ("layout", ctypes.c_int)]


class _Heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("x_token", ctypes.c_int64), ("x_head", ctypes.c_int64), ("y_token", ctypes.c_int64),
                ("y_head", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Table(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("ld", ctypes.c_int64), ("max_pages", ctypes.c_int32),
                ("batch", ctypes.c_int32)]


def _bad(func: str, detail: str) -> OrbqError:
    return OrbqError(-1, func, detail)


def _stream(t) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _heads_of(t, func: str, name: str):
    """A head tensor's checks: GPU, a known type, [tokens, heads, head_dim] with contiguous heads."""
    if not t.is_cuda:
        raise _bad(func, f"{name} must be on the GPU")
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise _bad(func, f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    if t.dtype not in _TYPES:
        raise _bad(func, f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return t


def _strides(t, *counts):
    # a dimension of one entry has no stride of its own: its entry count's worth is always aligned
    return tuple(0 if n <= 1 else s for n, s in zip(counts, t.stride()))


def _ints(t, like, count, func: str, name: str):
    if t.device != like.device or t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != count or \
            (count > 1 and t.stride(0) != 1):
        raise _bad(func, f"{name} must be contiguous int32 [{count}] on {like.device}")
    return t.data_ptr()


# ------------------------------------------------------------------------------------ rotary positions
@dataclass
class Rope:
    """dims: entries of a head that each axis turns (even; in order from entry 0; the rest of the head
    passes through).  freqs: float32 [sum(dims) / 2] on the GPU, radians per unit of position for each
    pair.  layout: "pairs" (2 i, 2 i + 1) or "halves" (i, i + sum(dims) / 2)."""
    dims: tuple
    freqs: "torch.Tensor"
    layout: str = "pairs"

    @classmethod
    def create(cls, dims, theta: float = 10000.0, layout: str = "pairs", device=None) -> "Rope":
        """Frequencies theta^(-2 i / dims[a]) for pair i of axis a."""
        f = torch.cat([theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in dims])
        return cls(tuple(dims), f.float().to(device or torch.device("cuda", torch.cuda.current_device())), layout)


def _rope(func, rope, positions, q, k, inverse, out):
    xs = [_heads_of(q, func, "q")] if k is None else [_heads_of(q, func, "q"), _heads_of(k, func, "k")]
    n, _, d = q.shape
    dims = rope.dims
    if not 1 <= len(dims) <= 4 or rope.layout not in LAYOUTS:
        raise _bad(func, f"{len(dims)} axes (1 to 4), layout {rope.layout!r} (one of {sorted(LAYOUTS)})")
    if len(xs) == 2 and (k.shape[0] != n or k.shape[2] != d or k.dtype != q.dtype or k.device != q.device):
        raise _bad(func, "q and k must agree in tokens, head_dim, type and device")
    if positions.device != q.device or positions.dtype != torch.float32 or positions.dim() != 2 or \
            positions.shape[1] != len(dims) or not positions.is_contiguous():
        raise _bad(func, f"positions must be contiguous float32 [tokens, {len(dims)}] on {q.device}")
    f = rope.freqs
    if f.device != q.device or f.dtype != torch.float32 or f.numel() != sum(dims) // 2 or not f.is_contiguous():
        raise _bad(func, f"freqs must be contiguous float32 [{sum(dims) // 2}] on {q.device}")
    if out is None:
        ys = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs]
    else:
        ys = [_heads_of(y, func, "out") for y in (out if isinstance(out, (tuple, list)) else (out,))]
        if len(ys) != len(xs) or any(x.shape != y.shape or x.dtype != y.dtype or x.device != y.device
                                     for x, y in zip(xs, ys)):
            raise _bad(func, "out must have the inputs' shapes, types and device")
    t = (_Heads * 2)()
    for i, (x, y) in enumerate(zip(xs, ys)):
        h = x.shape[1]
        t[i] = _Heads(x.data_ptr(), y.data_ptr(), h, *_strides(x, n, h), *_strides(y, n, h))
    r = _Rope(len(dims), (ctypes.c_int32 * 4)(*dims), f.data_ptr(), LAYOUTS[rope.layout])
    st = load().orbq_rope_apply(ctypes.byref(r), positions.data_ptr(), positions.shape[0], n, d, t, len(xs),
                                _TYPES[q.dtype], inverse, _stream(q))
    if st:
        _check(st, "orbq_rope_apply")
    return ys[0] if len(ys) == 1 else tuple(ys)


def rope(rope: Rope, positions, q, k=None, out=None):
    """q (and k, in the same launch) [tokens, heads, head_dim] turned by their positions float32
    [tokens or a divisor of it, axes].  out: where to write (the inputs themselves: in place)."""
    return _rope("rope", rope, positions, q, k, 0, out)


def rope_backward(rope: Rope, positions, dq, dk=None, out=None):
    """Gradients of rope's inputs from those of its outputs (the transposed map)."""
    return _rope("rope_backward", rope, positions, dq, dk, 1, out)


# ------------------------------------------------------------------------------------------ the cache
@dataclass
class KVCache:
    """k_codes int8 [pages, kv_heads, page_tokens, head_dim], v_codes int8 [pages, kv_heads, head_dim,
    page_tokens], k_scales and v_scales float32 [pages, kv_heads], all contiguous on one GPU."""
    k_codes: "torch.Tensor"
    v_codes: "torch.Tensor"
    k_scales: "torch.Tensor"
    v_scales: "torch.Tensor"

    @classmethod
    def create(cls, num_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device=None) -> "KVCache":
        dev = device or torch.device("cuda", torch.cuda.current_device())
        code = lambda *s: torch.empty(s, dtype=torch.int8, device=dev)  # noqa: E731
        scale = lambda: torch.empty((num_pages, kv_heads), dtype=torch.float32, device=dev)  # noqa: E731
        return cls(code(num_pages, kv_heads, page_tokens, head_dim), code(num_pages, kv_heads, head_dim, page_tokens),
                   scale(), scale())

    @property
    def page_tokens(self) -> int:
        return self.k_codes.shape[2]

    def struct(self, func: str) -> _Cache:
        k, v, ks, vs = self.k_codes, self.v_codes, self.k_scales, self.v_scales
        if k.dim() != 4:
            raise _bad(func, "k_codes must be [pages, kv_heads, page_tokens, head_dim]")
        n, h, t, d = k.shape
        if v.shape != (n, h, d, t) or ks.shape != (n, h) or vs.shape != (n, h):
            raise _bad(func, "the cache's tensors do not fit each other")
        if k.dtype != torch.int8 or v.dtype != torch.int8 or ks.dtype != torch.float32 or vs.dtype != torch.float32:
            raise _bad(func, "codes must be int8 and scales float32")
        if not (k.is_cuda and k.device == v.device == ks.device == vs.device):
            raise _bad(func, "the cache must be on one GPU")
        if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
            raise _bad(func, "the cache's tensors must be contiguous")
        return _Cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n, h, t, d)


def _table(table, cache, func: str) -> _Table:
    if table.device != cache.k_codes.device or table.dtype != torch.int32 or table.dim() != 2 or \
            (table.shape[1] > 1 and table.stride(1) != 1):
        raise _bad(func, f"table must be int32 [batch, pages] with contiguous rows on {cache.k_codes.device}")
    b, p = table.shape
    return _Table(table.data_ptr(), table.stride(0) if b > 1 else p, p, b)


def _moved(func, cache, k, v, table, first, cu, most):
    c, t = cache.struct(func), _table(table, cache, func)
    k, v = _heads_of(k, func, "k"), _heads_of(v, func, "v")
    n, h, d = k.shape
    if v.shape != k.shape or v.dtype != k.dtype or k.device != v.device or k.device != cache.k_codes.device or \
            h != c.kv_heads or d != c.head_dim:
        raise _bad(func, f"k and v must be [tokens, {c.kv_heads}, {c.head_dim}] of one type on the cache's device")
    first = _ints(first, k, t.batch, func, "positions")
    cu = 0 if cu is None else _ints(cu, k, t.batch + 1, func, "cu")
    if most is None:
        most = n if cu else n // max(1, t.batch)
    return (ctypes.byref(c), ctypes.byref(t), first, cu, n, most, k.data_ptr(), *_strides(k, n, h), v.data_ptr(),
            *_strides(v, n, h), _TYPES[k.dtype], _stream(k))


def kv_append(cache: KVCache, k, v, table, start, cu=None, max_new=None) -> None:
    """Quantises k, v [total, kv_heads, head_dim] and writes them behind the start[b] tokens that sequence b
    holds.  table int32 [batch, pages]; start int32 [batch]; cu int32 [batch + 1]: rows of each sequence (None:
    equal shares); max_new: no sequence has more (None: the most there can be)."""
    st = load().orbq_kv_append(*_moved("kv_append", cache, k, v, table, start, cu, max_new))
    if st:
        _check(st, "orbq_kv_append")


def kv_read(cache: KVCache, table, first, cu, total: int, max_tokens=None, dtype=torch.bfloat16, out=None):
    """(k, v) [total, kv_heads, head_dim] of tokens first[b] .. of each sequence, cu as in kv_append."""
    if out is None:
        shape = (total, cache.k_codes.shape[1], cache.k_codes.shape[3])
        out = tuple(torch.empty(shape, dtype=dtype, device=cache.k_codes.device) for _ in range(2))
    elif out[0].shape[0] != total:
        raise _bad("kv_read", f"out must have {total} tokens")
    st = load().orbq_kv_read(*_moved("kv_read", cache, out[0], out[1], table, first, cu, max_tokens))
    if st:
        _check(st, "orbq_kv_read")
    return out


# ---------------------------------------------------------------------------------------- attention
def kv_attention_workspace_bytes(cache: KVCache, batch: int, total: int, max_new: int, heads: int, max_len: int,
                                 causal_block: int = 0, window: int = 0) -> int:
    c = cache.struct("kv_attention")
    return int(load().orbq_kv_attention_workspace_bytes(ctypes.byref(c), batch, total, max_new, heads, max_len,
                                                        causal_block, window))


def kv_attention(cache: KVCache, q, table, lens, cu=None, max_new=None, causal_block: int = 0, window: int = 0,
                 scale=None, max_len=None, out=None, lse=None, workspace=None):
    """Attention of packed queries q [total, heads, head_dim] (bf16 or f16) over the cache; query i of the n of
    sequence b stands at position lens[b] - n + i.  causal_block: 0 none, 1 causal, tokens a frame: each frame
    sees itself and earlier ones.  window: at most that many of the latest visible tokens (0: all).  scale:
    1 / sqrt(head_dim) if None.  lse: float32 [total, heads] to receive the logarithms of the sums.
    max_len: expected bound of lens (None: what the table holds); it only guides how the work is split."""
    func = "kv_attention"
    c, t = cache.struct(func), _table(table, cache, func)
    q = _heads_of(q, func, "q")
    n, h, d = q.shape
    if q.device != cache.k_codes.device or d != c.head_dim:
        raise _bad(func, f"q must be [tokens, heads, {c.head_dim}] on the cache's device")
    lens = _ints(lens, q, t.batch, func, "lens")
    cu = 0 if cu is None else _ints(cu, q, t.batch + 1, func, "cu")
    if max_new is None:
        max_new = n if cu else n // max(1, t.batch)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device:
        raise _bad(func, "out must have q's shape, type and device")
    else:
        _heads_of(out, func, "out")
    if lse is not None and (lse.shape != (n, h) or lse.dtype != torch.float32 or lse.device != q.device or
                            not lse.is_contiguous()):
        raise _bad(func, f"lse must be contiguous float32 [{n}, {h}] on {q.device}")
    held = t.max_pages * c.page_tokens
    max_len = held if max_len is None else min(max_len, held)
    lib = load()
    if workspace is None:
        need = lib.orbq_kv_attention_workspace_bytes(ctypes.byref(c), t.batch, n, max_new, h, max_len, causal_block, window)
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device) if need else None
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = lib.orbq_kv_attention(ctypes.byref(c), ctypes.byref(t), lens, cu, n, max_new, max_len, q.data_ptr(),
                               *_strides(q, n, h), h, out.data_ptr(), *_strides(out, n, h),
                               0 if lse is None else lse.data_ptr(), _TYPES[q.dtype],
                               d ** -0.5 if scale is None else scale, causal_block, window, ws, ws_bytes, _stream(q))
    if st:
        _check(st, "orbq_kv_attention")
    return out
