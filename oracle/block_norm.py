"""Plain float64 oracle of the norms around a block and of their gradients, written from the formulas, row by row."""
from __future__ import annotations

import numpy as np


def groups_of(n: int, groups: int, cu=None) -> list:
    """Rows of each group."""
    if cu is None:
        return [range(n // groups * g, n // groups * (g + 1)) for g in range(groups)]
    return [range(cu[g], cu[g + 1]) for g in range(groups)]


def unit(v: np.ndarray, kind, eps: float):
    """(v normalised, the factor)"""
    if kind is None:
        return v, 1.0
    c = v - v.mean() if kind == "layer" else v
    f = 1.0 / np.sqrt((c * c).mean() + eps)
    return c * f, f


def row_of(v, g: int, default: float):
    """Row of group g of a vector [d], [1, d] or [groups, d]."""
    if v is None:
        return default
    return v if v.ndim == 1 else v[g if v.shape[0] > 1 else 0]


def stream(x, y, gate=None, post_weight=None, post=None, eps=1e-6, groups=1, cu=None) -> np.ndarray:
    """r = x + gate u; NaN where no group has the row."""
    r = np.full(x.shape, np.nan)
    w = 1.0 if post_weight is None else post_weight
    for g, rows in enumerate(groups_of(len(x), groups, cu)):
        for i in rows:
            r[i] = x[i] + row_of(gate, g, 1.0) * unit(y[i], post, eps)[0] * w
    return r


def normed(r, weight=None, scale=None, shift=None, norm="layer", eps=1e-6, groups=1, cu=None) -> np.ndarray:
    """h = norm(r) weight (1 + scale) + shift; NaN where no group has the row."""
    h = np.full(r.shape, np.nan)
    w = 1.0 if weight is None else weight
    for g, rows in enumerate(groups_of(len(r), groups, cu)):
        for i in rows:
            h[i] = unit(r[i], norm, eps)[0] * w * (1.0 + row_of(scale, g, 0.0)) + row_of(shift, g, 0.0)
    return h


def through_norm(v, t, kind, eps: float) -> np.ndarray:
    """Gradient of v from t, that of unit(v)."""
    if kind is None:
        return t
    z, f = unit(v, kind, eps)
    return f * (t - (t.mean() if kind == "layer" else 0.0) - z * (t * z).mean())


def gradients(r, dr, dh, y=None, gate=None, weight=None, scale=None, post_weight=None, norm="layer", post=None, eps=1e-6,
              post_eps=1e-6, groups=1, cu=None) -> dict:
    """Gradients of x, y (rows) and of gate, scale, shift (a row for each group), weight, post_weight (one row)."""
    n, d = r.shape
    w, pw = 1.0 if weight is None else weight, 1.0 if post_weight is None else post_weight
    out = {"x": np.zeros((n, d)), "y": np.zeros((n, d)), "weight": np.zeros(d), "post_weight": np.zeros(d)}
    out.update({a: np.zeros((groups, d)) for a in ("gate", "scale", "shift")})
    for g, rows in enumerate(groups_of(n, groups, cu)):
        s, c = 1.0 + row_of(scale, g, 0.0), row_of(gate, g, 1.0)
        for i in rows:
            at = np.zeros(d) if dr is None else dr[i].copy()
            if norm is not None:
                z, _ = unit(r[i], norm, eps)
                out["weight"] += dh[i] * s * z
                out["scale"][g] += dh[i] * w * z
                out["shift"][g] += dh[i]
                at += through_norm(r[i], dh[i] * w * s, norm, eps)
            out["x"][i] = at
            if y is None:
                continue
            z, _ = unit(y[i], post, post_eps)
            out["gate"][g] += at * z * pw
            out["post_weight"] += at * c * z
            out["y"][i] = through_norm(y[i], at * c * pw, post, post_eps)
    return out
