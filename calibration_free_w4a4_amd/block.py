"""Binding of the norms around a block (include/orbq.h says what they compute).  As elsewhere in this package the
functions only check and marshal arguments; the work is liborbq's HIP kernels.

    x, h = block_norm(x, y, gate=gate, scale=scale, shift=shift)     # x + gate y, and its modulated layer norm
    x, h = block_norm(x, y, weight=w1, post_weight=w0, norm="rms", post="rms")
    _, h = block_norm(x, scale=scale, shift=shift)                   # before the first branch: no y

Rows are tokens: x, y [n, d] with any row stride.  gate, scale and shift are [groups, d], a row for each sample whose
tokens follow one another (n / groups each, or as cu int32 [groups + 1] says), or [d] or [1, d] for all.

Gradients: block_norm is part of the autograd graph.  A call that is given `out` writes it and records nothing.
"""
from __future__ import annotations

import collections
import struct

from . import OrbqError, _check, load

__all__ = ["block_norm", "block_norm_backward", "NormGrads"]

torch = None       # with the first call: the package can be imported, with all its names, where there is none
_TYPES = {}
_Normed = None     # the autograd function

NORMS = {None: 0, "none": 0, "layer": 1, "rms": 2}   # orbq_norm_kind
_NORMS = struct.Struct("<2i2f5Q3q2iQi4x")            # orbq_norms
_GRADS = struct.Struct("<3Q3q2Q")                    # orbq_norms_grads

NormGrads = collections.namedtuple("NormGrads", "x y gate weight scale shift post_weight")
NormGrads.__doc__ = "Gradients of block_norm's inputs; None for one that is not there or not asked for."


def _need_torch() -> None:
    global torch, _Normed
    if torch is not None:
        return
    import torch as t
    from torch.autograd.function import once_differentiable

    class Normed(t.autograd.Function):
        @staticmethod
        def forward(ctx, func, dtype, how, x, y, gate, weight, scale, shift, post_weight):
            r, h = _forward(func, x, y, gate, weight, scale, shift, post_weight, dtype, None, **how)
            ctx.how = how
            ctx.save_for_backward(r, y, gate, weight, scale, shift, post_weight)
            ctx.set_materialize_grads(False)
            return h if y is None else r if h is None else (r, h)

        @staticmethod
        @once_differentiable
        def backward(ctx, *d):
            r, y, gate, weight, scale, shift, post_weight = ctx.saved_tensors
            how = dict(ctx.how)
            dr, dh = (None, d[0]) if y is None else d if len(d) == 2 else (d[0], None)
            needed = ctx.needs_input_grad[3:]
            if dr is None and dh is None:
                return (None,) * 10
            if dh is None:      # nothing came of h
                how["norm"], weight, scale, shift = None, None, None, None
            return (None, None, None) + tuple(_backward("block_norm", r, dh, dr, y, gate, weight, scale, shift, post_weight,
                                                        needed, None, **how))

    _TYPES.update({t.float32: 0, t.bfloat16: 1, t.float16: 2})
    _Normed = Normed
    torch = t


def _bad(func: str, detail: str) -> OrbqError:
    return OrbqError(-1, func, detail)


def _type(t, func: str, name: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        raise _bad(func, f"{name} must be float32, bfloat16 or float16 on the GPU, got {t.dtype} on {t.device}")
    return code


def _rows(t, like, func: str, name: str):
    """(address, row stride) of rows [n, d] shaped as `like` is."""
    if t.shape != like.shape or t.get_device() != like.get_device():
        raise _bad(func, f"{name} must be {list(like.shape)} on {like.device}")
    a, b = t.stride()
    if b != 1 and t.shape[1] > 1:
        raise _bad(func, f"{name} must have contiguous rows")
    return t.data_ptr(), a if t.shape[0] > 1 else 0


def _packed(x, y, gate, weight, scale, shift, post_weight, norm, post, eps, post_eps, cu, func):
    """(the packed orbq_norms, groups)"""
    n, d = x.shape
    dev = x.get_device()
    if norm not in NORMS or post not in NORMS:
        raise _bad(func, f"norm {norm!r}, post {post!r} (each one of 'layer', 'rms' or None)")
    if cu is not None:
        if cu.dtype != torch.int32 or cu.get_device() != dev or cu.dim() != 1 or cu.numel() < 2 or not cu.is_contiguous():
            raise _bad(func, f"cu must be contiguous int32 [groups + 1] on cuda:{dev}")
        groups = cu.numel() - 1
    else:
        groups = max([1] + [v.shape[0] for v in (gate, scale, shift) if v is not None and v.dim() == 2])
    at, mod = [], None
    for v, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
        if v is None:
            at += [(0, 0)]
            continue
        if v.shape not in ((d,), (1, d), (groups, d)) or v.get_device() != dev or (v.stride(-1) != 1 and d > 1):
            raise _bad(func, f"{name} must be [{d}] or [{groups}, {d}] with contiguous rows on cuda:{dev}, got {list(v.shape)}")
        if mod is not None and v.dtype != mod:
            raise _bad(func, "gate, scale and shift must be of one type")
        mod = v.dtype
        _type(v, func, name)
        at += [(v.data_ptr(), v.stride(0) if v.dim() == 2 and v.shape[0] > 1 else 0)]
    for v, name in ((weight, "weight"), (post_weight, "post_weight")):
        if v is not None and (v.shape != (d,) or v.get_device() != dev or (v.stride(0) != 1 and d > 1)):
            raise _bad(func, f"{name} must be contiguous [{d}] on cuda:{dev}")
    if weight is not None and post_weight is not None and weight.dtype != post_weight.dtype:
        raise _bad(func, "weight and post_weight must be of one type")
    w = weight if weight is not None else post_weight
    wtype = 0 if w is None else _type(w, func, "weight")
    address = lambda v: 0 if v is None else v.data_ptr()  # noqa: E731
    return _NORMS.pack(NORMS[norm], NORMS[post], eps, eps if post_eps is None else post_eps, address(weight), address(post_weight),
                       at[0][0], at[1][0], at[2][0], at[0][1], at[1][1], at[2][1], wtype, 0 if mod is None else _TYPES[mod],
                       address(cu), groups), groups


def _checked(x, y, func: str):
    """Types of the stream and of the branch that is there."""
    if x.dim() != 2:
        raise _bad(func, "x must be [rows, d]")
    code = _type(x, func, "x")
    return code, code if y is None else _type(y, func, "y")


def _forward(func, x, y, gate, weight, scale, shift, post_weight, dtype, out, norm, post, eps, post_eps, cu):
    code, branch = _checked(x, y, func)
    dev = x.get_device()
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _forward(func, x, y, gate, weight, scale, shift, post_weight, dtype, out, norm, post, eps, post_eps, cu)
    if dtype is not None and NORMS.get(norm):
        if dtype not in _TYPES or (y is not None and y.dtype != dtype):
            raise _bad(func, f"h cannot be {dtype}: one of the three types, and y's where there is a y")
        branch = _TYPES[dtype]
    norms, _ = _packed(x, y, gate, weight, scale, shift, post_weight, norm, post, eps, post_eps, cu, func)
    xp, xld = _rows(x, x, func, "x")
    yp, yld = (0, 0) if y is None else _rows(y, x, func, "y")
    n, d = x.shape
    h_type = dtype or (x if y is None else y).dtype
    if out is None:
        r = None if y is None else torch.empty((n, d), dtype=x.dtype, device=x.device)
        h = torch.empty((n, d), dtype=h_type, device=x.device) if NORMS[norm] else None
    else:
        r, h = out
        if y is None:
            r = None
        elif r is not None and r.dtype != x.dtype:
            raise _bad(func, f"r must be {x.dtype}")
        if NORMS[norm] and (h is None or h.dtype != h_type):
            raise _bad(func, f"h must be {h_type}")
        h = h if NORMS[norm] else None
    rp, rld = (0, 0) if r is None else _rows(r, x, func, "r")
    hp, hld = (0, 0) if h is None else _rows(h, x, func, "h")
    if n:
        st = load().orbq_block_norm(norms, n, d, xp, xld, yp, yld, rp, rld, hp, hld, code, branch,
                                    torch._C._cuda_getCurrentRawStream(dev))
        if st:
            _check(st, "orbq_block_norm")
    return (x if y is None else r), h


def block_norm(x, y=None, gate=None, weight=None, scale=None, shift=None, post_weight=None, norm="layer", post=None,
               eps: float = 1e-6, post_eps=None, cu=None, dtype=None, out=None):
    """(r, h): the stream r = x + gate * u, u = y or post(y) * post_weight, and the next branch's input
    h = norm(r) * weight * (1 + scale) + shift.  Without y, r is x; with norm None, h is None.
    norm, post: "layer", "rms" or None.  eps: of the norms (post_eps: of post, if another).  dtype: of h (None: that of y,
    or of x).  out: (r, h) to write; (x, h) writes r in place.  Rows outside cu's groups are left alone."""
    _need_torch()
    func = "block_norm"
    how = dict(norm=norm, post=post, eps=eps, post_eps=post_eps, cu=cu)
    if out is None and torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                                       for t in (x, y, gate, weight, scale, shift, post_weight)):
        got = _Normed.apply(func, dtype, how, x, y, gate, weight, scale, shift, post_weight)
        return (x, got) if y is None else got if isinstance(got, tuple) else (got, None)
    return _forward(func, x, y, gate, weight, scale, shift, post_weight, dtype, out, **how)


def _backward(func, r, dh, dr, y, gate, weight, scale, shift, post_weight, needed, workspace, norm, post, eps, post_eps, cu):
    code, branch = _checked(r, y, func)
    dev = r.get_device()
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _backward(func, r, dh, dr, y, gate, weight, scale, shift, post_weight, needed, workspace, norm, post, eps,
                             post_eps, cu)
    norms, groups = _packed(r, y, gate, weight, scale, shift, post_weight, norm, post, eps, post_eps, cu, func)
    n, d = r.shape
    if dh is None and dr is None:
        raise _bad(func, "neither dh nor dr")
    if dh is not None:
        branch = _type(dh, func, "dh")
        if y is not None and y.dtype != dh.dtype:
            raise _bad(func, "dh must have y's type")
    if dr is not None and dr.dtype != r.dtype:
        raise _bad(func, "dr must have r's type")
    given = (r, y, gate, weight, scale, shift, post_weight)
    got = [None if t is None or not need else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t, need in zip(given, needed)]
    if n == 0:
        return NormGrads(*[None if t is None else t.zero_() for t in got])
    flat = lambda t: t if t is None or t.stride(-1) == 1 or d == 1 else t.contiguous()  # noqa: E731  an expanded gradient
    dh, dr = flat(dh), flat(dr)
    rp, rld = _rows(r, r, func, "r")
    yp, yld = (0, 0) if y is None else _rows(y, r, func, "y")
    drp, drld = (0, 0) if dr is None else _rows(dr, r, func, "dr")
    dhp, dhld = (0, 0) if dh is None else _rows(dh, r, func, "dh")
    address = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    # a vector that the groups share has one gradient, the sum of theirs
    apart = lambda t: 0 if t is None or t.dim() == 1 or (t.shape[0] == 1 and groups > 1) else d  # noqa: E731
    dx, dy, dgate, dweight, dscale, dshift, dpost = got
    ws, ws_bytes = 0, 0
    if any(t is not None for t in got[2:]):
        if workspace is None:
            ws_bytes = load().orbq_block_norm_backward_workspace_bytes(n, d, groups)
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=r.device)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise _bad(func, f"workspace must be contiguous on cuda:{dev}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    grads = _GRADS.pack(address(dgate), address(dscale), address(dshift), apart(dgate), apart(dscale), apart(dshift),
                        address(dweight), address(dpost))
    st = load().orbq_block_norm_backward(norms, n, d, rp, rld, yp, yld, drp, drld, dhp, dhld, address(dx), d, address(dy), d, grads,
                                         code, branch, ws, ws_bytes, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "orbq_block_norm_backward")
    return NormGrads(*got)


def block_norm_backward(r, dh, dr=None, y=None, gate=None, weight=None, scale=None, shift=None, post_weight=None, norm="layer",
                        post=None, eps: float = 1e-6, post_eps=None, cu=None, workspace=None) -> NormGrads:
    """Gradients of block_norm's inputs from those of its outputs, dr (None: zero) and dh (None with norm None).  r is the
    stream that the forward pass gave (x where there was no y); the other arguments as there.  Each vector that is
    given gets its gradient, of its own shape and type."""
    _need_torch()
    return _backward("block_norm_backward", r, dh, dr, y, gate, weight, scale, shift, post_weight, (True,) * 7, workspace,
                     norm=norm, post=post, eps=eps, post_eps=post_eps, cu=cu)
