"""The epilogue oracle: against values written out by hand."""
import math

import numpy as np

from oracle.epilogue import epilogue


def test_by_hand():
    y = np.array([[1.0, -2.0], [0.5, 3.0], [4.0, 0.0]])
    bias, gate, res = np.array([1.0, 2.0]), np.array([[2.0, -1.0], [0.0, 5.0]]), np.array([[10.0, 20.0], [30.0, 40.0], [50.0, 60.0]])
    want = np.array([[4.0 + 10, 0.0 + 20], [3.0 + 30, -5.0 + 40], [0.0 + 50, 10.0 + 60]])
    assert np.allclose(epilogue(y, "none", bias, gate, res, 2, [0, 2, 3]), want)
    assert np.allclose(epilogue(y[:2], "none", bias, gate, res[:2], 2), [[14.0, 20.0], [30.0, 65.0]])
    got = epilogue(y, "gelu_erf", None, None, None, 2, [1, 1, 2])
    assert np.isnan(got[[0, 2]]).all()
    assert abs(got[1, 0] - 0.5 * 0.5 * (1 + math.erf(0.5 / math.sqrt(2)))) < 1e-12
    one = epilogue(y, "gelu_tanh", None, gate[0])
    x = 3.0
    assert abs(one[1, 1] + 0.5 * x * (1 + math.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))) < 1e-12
