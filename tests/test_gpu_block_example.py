"""examples/video_transformer_block.py: the operators together.  Each call that a step makes is recorded with its inputs and its
result, and held to the definition in 64 bits from these; tolerances as in the operators' own tests (the products' from their
codes, whose quantizer has its own)."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from oracle import attention as oa
from oracle import block_norm as ob
from oracle.epilogue import epilogue
from tests.gpu_common import log, torch_mod
from tests.test_gpu_block_norm import close, off, per_row

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = 2.0 ** -24
NAMES = ("block_norm", "linear", "linear_a16", "kv_append_rope", "kv_attention")


@pytest.fixture(scope="module")
def example():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("block_example", os.path.join(ROOT, "examples", "video_transformer_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


@pytest.fixture
def calls(example, monkeypatch):
    """[(name, positional and keyword inputs as they were, result as it was)] of the calls made."""
    torch, made = torch_mod(), []
    copy = lambda v: v.clone() if isinstance(v, torch.Tensor) else v  # noqa: E731

    def record(name, func):
        def call(*a, **kw):
            given = [copy(v) for v in a], {k: copy(v) for k, v in kw.items() if k != "out"}
            got = func(*a, **kw)
            made.append((name, *given, tuple(copy(v) for v in got) if isinstance(got, tuple) else copy(got)))
            return got
        return call
    for name in NAMES:
        monkeypatch.setattr(example.orbq, name, record(name, getattr(example.orbq, name)))
    return made


def check_norm(x, got, y=None, gate=None, scale=None, shift=None, dtype=None):
    n, d = x.shape
    r, h = got
    groups = len(scale)
    x, y64, gate, scale, shift = (host(t) for t in (x, y, gate, scale, shift))
    if y is None:
        assert np.array_equal(host(r), x)
    else:
        c = np.abs(per_row(gate, groups, n, None, 1.0))
        close(r, ob.stream(x, y64, gate, groups=groups), 4 * E * (c * np.abs(y64) + np.abs(x)), "f32", "r")
    r = host(r)
    z = np.stack([ob.unit(row, "layer", 1e-6)[0] for row in r])
    c = 1 + np.abs(per_row(scale, groups, n, None, 0.0))
    close(h, ob.normed(r, None, scale, shift, groups=groups), c * (off(r, "layer", 1e-6) + 4 * E * np.abs(z)) +
          4 * E * np.abs(per_row(shift, groups, n, None, 0.0)), "bf16", "h")


def check_product(orbq, func, x, rot, rest, got, bias, act="none", gate=None, residual=None, out_dtype=None):
    d = x.shape[1]
    w_codes, w_norms, cb = rest[-3:]
    decode = lambda codes: oracle.decode_lut_bf16(cb.centroids)[oracle.unpack_codes(codes.cpu().numpy(), cb.bits, d)]  # noqa: E731
    b = decode(w_codes) * host(w_norms)[:, None]
    if func == "linear_a16":
        perm, signs = rot.perm.cpu().numpy(), rot.signs.cpu().numpy()
        a, rel = host(x) @ oracle.rpbh_matrix(d, rot.block, perm, signs).T, 2.0 ** -8 + (d / 8 + 40) * E
    else:
        codes, s = orbq.rpbh_quantize(x, rot, cb)
        a, rel = decode(codes) * host(s)[:, None], (d / 8 + 36) * E
    product, bias, gate, residual = a @ b.T, host(bias), host(gate), host(residual)
    groups = 1 if gate is None else len(gate)
    pre = product + bias
    tol = rel * (np.abs(a) @ np.abs(b).T) + 2 * E * (np.abs(bias) + np.abs(pre))
    if act != "none":
        tol = 1.13 * tol + 6e-7 * np.abs(pre)
    tol *= np.abs(per_row(gate, groups, len(pre), None, 1.0))
    want = epilogue(product, act, bias, gate, residual, groups)
    tol += 2 * E * (np.abs(want) + (0 if residual is None else 2 * np.abs(residual)))
    close(got, want, tol, "bf16" if got.dtype == torch_mod().bfloat16 else "f32", func)


def check_append(cache, rope, positions, q, k, v, table, start, got, q_weight, k_weight):
    """cache as it is behind the call."""
    n, batch, page = len(k), len(table), cache.page_tokens
    each = n // batch
    pos = np.tile(host(positions), (batch, 1))
    rel = 1.3e-6

    def turned(x, w):
        x = host(x)
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * host(w)
        a, b = oa.rope_pairs(rope.dims, "pairs")
        size = np.abs(x)
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return oa.rope(x, rope.dims, host(rope.freqs).astype(np.float32), pos.astype(np.float32), "pairs"), size
    want, size = turned(q, q_weight)
    close(got, want, rel * size, "bf16", "q")
    at = host(start).astype(int).repeat(each) + np.tile(np.arange(each), batch)
    pages = table.cpu().numpy()[np.arange(batch).repeat(each), at // page]
    k64, size = turned(k, k_weight)
    for codes, scales, x, err in ((host(cache.k_codes)[pages, :, at % page], host(cache.k_scales)[pages], k64, rel * size),
                                  (host(cache.v_codes)[pages, :, :, at % page], host(cache.v_scales)[pages], host(v), 0.0)):
        s = scales[..., None]
        # half a step of the page's scale, which came from the same entries (2 rel), and 1 / scale's and the product's roundings
        assert np.all(np.abs(codes * s - x) <= 0.5 * s + err + 127 * s * (2 * rel if np.ndim(err) else 4 * E))


@pytest.mark.parametrize("clips,chunk", [(1, 1), (2, 2), (3, 1)])
def test_steps(example, calls, clips, chunk):
    torch, orbq = torch_mod(), example.orbq
    h, w, frames, d, heads, hidden = 5, 7, 3, 256, 2, 640
    block = example.StreamingBlock(d, heads, hidden, clips, frames * h * w, h * w)
    gen = torch.Generator(device="cuda").manual_seed(clips)
    held = 0
    for f in range(0, frames, chunk):
        fr = range(f, min(f + chunk, frames))
        n = len(fr) * h * w
        x = 2 * torch.randn((clips * n, d), generator=gen, device="cuda") + 0.3
        condition = torch.randn((clips, d), generator=gen, device="cuda").bfloat16()
        pos = example.grid_positions(fr, h, w)
        del calls[:]
        got = block.step(x, pos, condition)
        assert got is x and [c[0] for c in calls] == ["linear_a16", "block_norm", "linear", "kv_append_rope", "kv_attention", "linear",
                                                      "block_norm", "linear", "linear"]
        for name, a, kw, out in list(calls):
            log(f"clips {clips} frames {fr}: {name} {[tuple(t.shape) for t in a if isinstance(t, torch.Tensor)]}")
            if name == "block_norm":
                check_norm(a[0], out, *a[1:], **kw)
            elif name == "kv_append_rope":
                check_append(block.cache, *a[1:], out, **kw)
            elif name == "kv_attention":
                q = host(a[1]).reshape(clips, n, heads, block.hd)
                for b in range(clips):
                    table, (kc, vc, ks, vs) = block.table[b].cpu().numpy(), (
                        t.cpu().numpy() for t in (block.cache.k_codes, block.cache.v_codes, block.cache.k_scales, block.cache.v_scales))
                    keys, values = oa.kv_tokens(kc, ks, table, held + n, False), oa.kv_tokens(vc, vs, table, held + n, True)
                    want, _, spread = oa.attention(q[b], keys, values, h * w, 0, block.hd ** -0.5)
                    # as in tests/test_gpu_attention.py
                    eps = 2.0 ** -11 + 2.0 ** -17 + 2 * (block.hd + 8) * E * spread[..., 1:2]
                    tol = 2.0 ** -8 * np.abs(want) * (1 + eps) + eps * spread[..., 0:1] + len(keys) * E * spread[..., 2:3]
                    assert np.all(np.abs(host(out).reshape(clips, n, heads, block.hd)[b] - want) <= tol)
            else:
                check_product(orbq, name, a[0], a[1], a[2:], out, **kw)
        # the stream that came out is the last call's result, and the next step sees every clip's tokens
        assert torch.equal(x, calls[-1][3])
        held += n
        assert block.held.tolist() == [held] * clips


def test_captured_step(example):
    """A step as a graph: every replay appends behind what the caches hold by then and gives the eager step's bits."""
    torch = torch_mod()
    h, w, frames, d = 4, 4, 5, 256
    gen = torch.Generator(device="cuda").manual_seed(3)
    xs = torch.randn((frames, 2 * h * w, d), generator=gen, device="cuda")
    condition = torch.randn((2, d), generator=gen, device="cuda").bfloat16()
    pos = torch.stack([example.grid_positions(range(f, f + 1), h, w) for f in range(frames)])
    eager, captured = (example.StreamingBlock(d, 2, 384, 2, frames * h * w, h * w) for _ in range(2))
    want = [eager.step(x.clone(), p, condition) for x, p in zip(xs, pos)]
    x, p = torch.empty_like(xs[0]), torch.empty_like(pos[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(xs[0])
        p.copy_(pos[0])
        assert torch.equal(captured.step(x, p, condition), want[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(x, p, condition)
    for f in range(1, frames):
        x.copy_(xs[f])
        p.copy_(pos[f])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[f])
    # the tokens that the caches hold; what lies behind them nobody has written
    total = 2 * frames * h * w
    cu = torch.tensor([0, total // 2, total], dtype=torch.int32, device="cuda")
    held = [example.orbq.kv_read(b.cache, b.table, torch.zeros_like(b.held), cu, total) for b in (eager, captured)]
    assert all(torch.equal(a, b) for a, b in zip(*held))


def test_command(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["block", "--width-d", "256", "--heads", "2", "--hidden", "384", "--clips", "2", "--frames", "2",
                                     "--chunk", "1", "--height", "3", "--width", "5"])
    example.main()
    assert len(capsys.readouterr().out.splitlines()) == 2
