"""examples/streaming_video_attention.py: the operators together, step by step, against the same steps in
64 bits (projections through the library, whose parity has its own tests)."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_common import log, torch_mod

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("streaming_example", os.path.join(ROOT, "examples", "streaming_video_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("chunk", [1, 2])
def test_steps(example, chunk):
    torch = torch_mod()
    orbq = example.orbq
    h, w, frames, d, heads = 5, 7, 5, 256, 2
    layer = example.StreamingAttention(d, heads, frames * h * w, h * w)
    rng = np.random.default_rng(chunk)
    hd, page = layer.hd, layer.cache.page_tokens
    pages = layer.table.shape[1]
    kc, vc = np.zeros((pages, heads, page, hd), np.int8), np.zeros((pages, heads, hd, page), np.int8)
    ks, vs = np.zeros((pages, heads), np.float32), np.zeros((pages, heads), np.float32)
    table, held = layer.table.cpu().numpy(), 0
    freqs = layer.rope.freqs.cpu().numpy()
    for f in range(0, frames, chunk):
        fr = range(f, min(f + chunk, frames))
        n = len(fr) * h * w
        x = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda().bfloat16()
        pos = example.grid_positions(fr, h, w)
        y = layer.step(x, pos)
        # the same in 64 bits, from the library's projection
        qkv = orbq.linear(x, layer.rot, layer.cb, *layer.qkv, layer.cb, out_dtype=torch.bfloat16).view(n, 3, heads, hd)
        q, k, v = (t.double().cpu().numpy() for t in qkv.unbind(1))
        bf16 = lambda a: torch.from_numpy(a).bfloat16().double().numpy()  # noqa: E731
        q, k = (bf16(oa.rope(t, layer.rope.dims, freqs, pos.cpu().numpy(), "pairs")) for t in (q, k))
        oa.kv_append(kc, vc, ks, vs, table, [held], [k.astype(np.float32)], [v.astype(np.float32)])
        held += n
        o, _, spread = oa.attention(q, oa.kv_tokens(kc, ks, table[0], held, False), oa.kv_tokens(vc, vs, table[0], held, True),
                                    h * w, 0, hd ** -0.5)
        want = orbq.linear(torch.from_numpy(o).bfloat16().cuda().reshape(n, d), layer.rot, layer.cb, *layer.out, layer.cb,
                           out_dtype=torch.bfloat16).float()
        # A rope result on a bf16 rounding boundary may go to the other side, and so may what follows: a few
        # units of bf16 in o.  The projection's 4-bit codes turn those into at most one code step for a few
        # of its inputs: 5 % of the output's norm is a fifth of what one step for all would be.
        err = (y.float() - want).norm() / want.norm()
        log(f"frames {fr}: rel {err.item():.2e}")
        assert err.item() < 0.05
        assert layer.held.item() == held
