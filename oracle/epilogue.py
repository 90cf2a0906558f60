"""What a block does behind a product, in float64: bias, activation, gate, residual (include/orbq.h, orbq_epilogue)."""
from __future__ import annotations

import numpy as np

from .activation import activation
from .block_norm import groups_of, row_of


def epilogue(product, act="none", bias=None, gate=None, residual=None, groups=1, cu=None) -> np.ndarray:
    """residual + gate[group of the row] act(product + bias); NaN where no group has the row."""
    y = np.asarray(product, np.float64)
    if bias is not None:
        y = y + bias
    y = activation(y, act)
    out = np.full(y.shape, np.nan)
    for g, rows in enumerate(groups_of(len(y), groups, cu)):
        for i in rows:
            out[i] = y[i] * row_of(gate, g, 1.0) + (0.0 if residual is None else residual[i])
    return out
