"""Row strides that the operators around a block's projections allow and models rarely have: rows that are one and the same, and rows
so far apart that their offsets pass 32 bits.  Results are those of the same values in contiguous tensors, bit for bit."""
import pytest

from tests.conftest import oracle_codebook
from tests.gpu_common import log, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def orbq():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import calibration_free_w4a4_amd as m
    m.load()
    return m


def normal(gen, *shape):
    return torch_mod().randn(shape, generator=gen, device="cuda")


@pytest.mark.parametrize("d", [96, 100, 1536, 4096])
def test_rows_that_are_one(orbq, d):
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 37
    x, y, dh, dr = (normal(gen, 1, d).bfloat16().expand(n, d) for _ in range(4))
    gate, scale, shift, w = (normal(gen, d) for _ in range(4))
    w = w.bfloat16()
    how = dict(gate=gate, scale=scale, shift=shift, weight=w, post_weight=w, norm="rms", post="layer")
    apart = orbq.block_norm(x.contiguous(), y.contiguous(), **how)
    got = orbq.block_norm(x, y, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, apart))
    got = orbq.block_norm_backward(x, dh, dr, y=y, **how)
    apart = orbq.block_norm_backward(x.contiguous(), dh.contiguous(), dr.contiguous(), y=y.contiguous(), **how)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, apart))
    # the gradient of a sum over rows is such a tensor
    leaf = x.contiguous().requires_grad_()
    r, h = orbq.block_norm(leaf, y, **how)
    (r.float().sum(0) @ normal(gen, d) + h.float().sum(0) @ normal(gen, d)).backward()
    assert bool(torch.isfinite(leaf.grad.float()).all())


def test_norm_rows_far_apart(orbq):
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(1)
    n, d, ld = 600, 136, (1 << 21) + 8      # 600 rows of 8 MiB: 5 GB
    far = torch.empty((n, ld), dtype=torch.float32, device="cuda")
    x, r = far[:, :d], far[:, d:2 * d]
    x.copy_(normal(gen, n, d))
    y = normal(gen, n, d)
    how = dict(gate=normal(gen, 3, d), scale=normal(gen, 3, d), shift=normal(gen, 3, d))
    want = orbq.block_norm(x.contiguous(), y, **how)
    h = far[:, 2 * d:3 * d]
    orbq.block_norm(x, y, out=(r, h), **how)
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])
    got = orbq.block_norm_backward(r, h, x, y=y, **how)
    for a, b in zip(got, orbq.block_norm_backward(want[0], want[1], x.contiguous(), y=y, **how)):
        assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("n,ld", [(64, 1 << 21), (4200, 1 << 19)])
def test_product_rows_far_apart(orbq, n, ld):
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(n)
    m, d = 200, 256
    cb = orbq.Codebook.from_centroids(d, 4, oracle_codebook(d, 4))
    code = lambda rows: torch.randint(0, 256, (rows, d // 2), generator=gen, device="cuda").to(torch.uint8)  # noqa: E731
    args = (code(n), normal(gen, n).abs(), cb, code(m), normal(gen, m).abs().bfloat16(), cb, d)
    far = torch.empty((n, ld), dtype=torch.bfloat16, device="cuda")
    y, res = far[:, :m], far[:, 256:256 + m]
    res.copy_(normal(gen, n, m))
    how = dict(bias=normal(gen, m), gate=normal(gen, 2, m), act="gelu_tanh")
    want = orbq.lut_gemm(*args, residual=res.contiguous(), **how)
    assert orbq.lut_gemm(*args, residual=res, out=y, **how) is y
    assert torch.equal(y, want)


def test_append_to_far_pages(orbq):
    """Pages beyond 4 GiB of codes."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(3)
    heads, page, d, pages = 8, 64, 128, 66000
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = (normal(gen, 100, heads, d).bfloat16() for _ in range(3))
    rope, pos = orbq.Rope.create((d,)), torch.arange(100, dtype=torch.float32, device="cuda")[:, None].contiguous()
    w = normal(gen, d)
    out = []
    for count, table in ((4, [[0, 1], [2, 3]]), (pages, [[65990, 2], [65999, 65998]])):
        cache = orbq.KVCache.create(count, heads, d, page)
        log(f"{count} pages")
        got = orbq.kv_append_rope(cache, rope, pos, q, k, v, ints(table), ints([0, 0]), cu=ints([0, 70, 100]), max_new=70, q_weight=w, k_weight=w)
        out.append((got,) + tuple(orbq.kv_read(cache, ints(table), ints([0, 0]), ints([0, 70, 100]), 100)))
    assert all(torch.equal(a, b) for a, b in zip(*out))
