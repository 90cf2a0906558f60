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
