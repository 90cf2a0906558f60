"""The attention-side operators on the GPU against the float64 oracle (oracle/attention.py).

Tolerances, from the arithmetic before any run:
  * rope: the angle loses 2^-26 of a turn (9.4e-8 rad), the polynomial and its argument 1.2e-7, the two
    products and their sum 1.8e-7, all relative to |a| + |b| of the pair: 5e-7 (|a| + |b|), and half a unit of
    the output type;
  * kv_append, kv_read: bit for bit (each step is one fp32 operation);
  * kv_attention: weights are rounded to f16 (2^-11 relative; below the normal range 2^-25 of the largest,
    counted twice, since the largest code of a block need not be 127), scores carry (d + 8) 2^-24 of sum
    |q| |k| scale, the exponent with its scale's logarithm (up to 50) and exp2 2^-17;
    relative to sum_j P_j |v_j|, plus half a unit of the output type.
"""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_common import log, torch_mod

pytestmark = pytest.mark.gpu
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def orbq():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import calibration_free_w4a4_amd as m
    m.load()
    return m


def dtype_of(name):
    torch = torch_mod()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def dev(x, name="f32"):
    """numpy -> GPU tensor of the type, and the float64 values it holds."""
    torch = torch_mod()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype_of(name)).cuda()
    return t, t.double().cpu().numpy()


def ints(v):
    torch = torch_mod()
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def strided(x, pad_heads, pad_d):
    """The same values as the middle of a wider tensor (as part of a fused projection)."""
    torch = torch_mod()
    n, h, d = x.shape
    big = torch.full((n, h + pad_heads, d + pad_d), float("nan"), dtype=x.dtype, device=x.device)
    view = big[:, pad_heads // 2:pad_heads // 2 + h, :d]
    view.copy_(x)
    return view


# ------------------------------------------------------------------------------------------- rope
def check_rope(got, x64, dims, freqs, pos, layout, inverse, name):
    want = oa.rope(x64, dims, freqs, pos, layout, inverse)
    a, b = oa.rope_pairs(dims, layout)
    size = np.zeros(x64.shape)
    size[..., a] = size[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    tol = 5e-7 * size + UNIT[name] * np.abs(want) * (1 + 1e-6) + LEAST[name]
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{(err / tol).max():.3g} of the tolerance at {np.unravel_index((err / tol).argmax(), err.shape)}"
    rest = sum(dims)
    assert np.array_equal(got.double().cpu().numpy()[..., rest:], x64[..., rest:])


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("n,qh,kh,d,dims", [
    (1, 12, 12, 128, (44, 42, 42)), (333, 5, 1, 128, (16, 56, 56)), (65, 3, 2, 64, (16, 24, 24)),
    (40, 2, 2, 256, (64, 64, 64)), (17, 3, 3, 72, (24, 24, 24)), (9, 1, 4, 6, (2, 2)), (5, 2, 1, 512, (512,)),
    (30, 7, 1, 96, (10, 20, 30, 4)), (2100, 24, 8, 128, (32, 48, 48))])
def test_rope(orbq, name, layout, n, qh, kh, d, dims):
    log(f"rope {name} {layout} n={n} heads {qh}/{kh} d={d} dims={dims}")
    rng = np.random.default_rng(n + d)
    pos = rng.uniform(-300, 300, (n, len(dims))).astype(np.float32)
    pos[: n // 2] = np.round(pos[: n // 2])
    r = orbq.Rope.create(dims, layout=layout)
    freqs = r.freqs.cpu().numpy()
    p, _ = dev(pos)
    q, q64 = dev(rng.standard_normal((n, qh, d)) * 3, name)
    k, k64 = dev(rng.standard_normal((n, kh, d)), name)
    for inverse, call in ((False, orbq.rope), (True, orbq.rope_backward)):
        yq, yk = call(r, p, q, k)
        check_rope(yq, q64, dims, freqs, pos, layout, inverse, name)
        check_rope(yk, k64, dims, freqs, pos, layout, inverse, name)
    # strided in, strided out, and in place: the same bits
    want = orbq.rope(r, p, q)
    for pad in ((4, 16), (2, 2)):        # 16-byte columns, and not
        qs, ys = strided(q, *pad), strided(q * 0, *pad)
        assert orbq.rope(r, p, qs, out=ys) is ys
        assert torch_mod().equal(ys, want)
        assert bool(torch_mod().isnan(ys._base[:, :, d:]).all())
        orbq.rope(r, p, qs, out=qs)
        assert torch_mod().equal(qs, ys)


def test_rope_far_positions_and_shared_grid(orbq):
    """Positions far along an axis stay as exact as near ones; a batch of grids shares one set."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    r = orbq.Rope.create((20, 12))
    pos = np.concatenate([rng.uniform(-2 ** 20, 2 ** 20, (50, 2)), [[16777216.0, -16777216.0], [0.0, 1e-3]]]).astype(np.float32)
    p, _ = dev(pos)
    x, x64 = dev(rng.standard_normal((len(pos), 3, 32)))
    check_rope(orbq.rope(r, p, x), x64, (20, 12), r.freqs.cpu().numpy(), pos, "pairs", False, "f32")
    y = orbq.rope(r, p, torch.cat([x, x, x]))
    assert torch.equal(y[:52], y[52:104]) and torch.equal(y[:52], y[104:])
    # not finite: only the pairs that hold it are lost
    x[3, 1, 7] = float("inf")
    x[4, 2, 0] = float("nan")
    z = orbq.rope(r, p, x)
    bad = ~torch.isfinite(z)
    want = torch.zeros_like(bad)
    want[3, 1, 6:8] = True
    want[4, 2, 0:2] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_gradient_by_differences(orbq, layout):
    """<dy, rope(x + e) - rope(x - e)> / 2 = <rope_backward(dy), e>: the map is linear, so the only error is
    fp32 rounding, 5e-7 of each product's size."""
    rng = np.random.default_rng(8)
    r = orbq.Rope.create((44, 42, 42), layout=layout)
    p, _ = dev(rng.integers(0, 60, (37, 3)))
    x, e, dy = (dev(rng.standard_normal((37, 4, 128)))[0] for _ in range(3))
    diff = (orbq.rope(r, p, x + e).double() - orbq.rope(r, p, x - e).double()) / 2
    lhs = (dy.double() * diff).sum((1, 2))
    rhs = (orbq.rope_backward(r, p, dy).double() * e.double()).sum((1, 2))
    tol = 4 * 5e-7 * (dy.double().abs().amax() * 2 * (x.abs() + e.abs()).double().sum((1, 2)))
    assert bool(((lhs - rhs).abs() <= tol).all())
    back = orbq.rope_backward(r, p, orbq.rope(r, p, x))
    assert (back - x).abs().max().item() <= 4 * 5e-7 * 2 * x.abs().max().item()


# ------------------------------------------------------------------------------------------ cache
def cache_of(orbq, rng, pages, heads, d, page):
    """A cache whose every byte is set: what is not written must stay as it is."""
    torch = torch_mod()
    c = orbq.KVCache.create(pages, heads, d, page)
    c.k_codes.copy_(torch.from_numpy(rng.integers(-127, 128, (pages, heads, page, d), dtype=np.int8)))
    c.v_codes.copy_(torch.from_numpy(rng.integers(-127, 128, (pages, heads, d, page), dtype=np.int8)))
    for s in (c.k_scales, c.v_scales):
        s.copy_(torch.from_numpy(np.exp(rng.uniform(-6, -3, (pages, heads))).astype(np.float32)))
    return c


def host(c):
    return [t.cpu().numpy().copy() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]


def table_of(rng, pages, lens, page, extra=0):
    per = [(n + page - 1) // page for n in lens]
    order = rng.permutation(pages)[: sum(per)]
    t = np.full((len(lens), max(1, max(per) + extra)), -1, np.int32)
    at = 0
    for b, k in enumerate(per):
        t[b, :k] = order[at:at + k]
        at += k
    return t


def compare_cache(c, want, table, lens, page):
    """Scales and the codes of held tokens bit for bit; blocks of nobody untouched."""
    got = host(c)
    owned = set(int(x) for x in table.ravel() if x >= 0)
    for g, w in zip(got, want):
        for pg in range(len(g)):
            if pg not in owned:
                assert np.array_equal(g[pg], w[pg], equal_nan=True), f"block {pg} of nobody was written"
    for b, n in enumerate(lens):
        for p in range((n + page - 1) // page):
            pg, m = int(table[b, p]), min(page, n - p * page)
            if pg < 0:
                continue
            assert np.array_equal(got[2][pg], want[2][pg]) and np.array_equal(got[3][pg], want[3][pg]), (b, p)
            assert np.array_equal(got[0][pg][:, :m], want[0][pg][:, :m]), (b, p)
            assert np.array_equal(got[1][pg][:, :, :m], want[1][pg][:, :, :m]), (b, p)


@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_and_read(orbq, name, d, page):
    torch = torch_mod()
    rng = np.random.default_rng(page + d)
    start = [0, 1, page - 1, page, 2 * page + 5, 7, 3]
    new = [2 * page + 3, 1, 1, page, 3 * page, 0, 2]
    heads = 3
    log(f"append {name} d={d} page={page}")
    lens = [a + b for a, b in zip(start, new)]
    pages = sum((n + page - 1) // page for n in lens) + 3
    table = table_of(rng, pages, lens, page, extra=1)
    c = cache_of(orbq, rng, pages, heads, d, page)
    want = host(c)
    cu = np.concatenate([[0], np.cumsum(new)])
    total = int(cu[-1])
    # rows of very different size, so that some blocks grow and some do not
    size = np.exp(rng.uniform(-4, 3, (total, 1, 1)))
    k, k64 = dev(rng.standard_normal((total, heads, d)) * size, name)
    v, v64 = dev(rng.standard_normal((total, heads, d)) * size, name)
    split = lambda x: [x[cu[b]:cu[b + 1]].astype(np.float32) for b in range(len(new))]  # noqa: E731
    oa.kv_append(*want, table, start, split(k64), split(v64))
    ks, vs = strided(k, 4, 16), strided(v, 2, 8)
    orbq.kv_append(c, ks, vs, ints(table), ints(start), cu=ints(cu), max_new=max(new))
    compare_cache(c, want, table, lens, page)
    # read back from a token inside the first block that was there before
    first = [max(0, s - 2) for s in start]
    n = [a - b for a, b in zip(lens, first)]
    cr = np.concatenate([[0], np.cumsum(n)])
    out = [strided(torch.zeros((int(cr[-1]), heads, d), dtype=k.dtype, device="cuda"), 2, 16) for _ in range(2)]
    orbq.kv_read(c, ints(table), ints(first), ints(cr), int(cr[-1]), max_tokens=max(n), out=out)
    for o, codes, scales, turned in ((out[0], want[0], want[2], False), (out[1], want[1], want[3], True)):
        for b in range(len(new)):
            # code * scale in fp32 is the float64 product rounded once
            w = oa.kv_tokens(codes, scales, table[b], lens[b], turned)[first[b]:].astype(np.float32)
            w = torch.from_numpy(w).to(k.dtype)
            assert torch.equal(o[cr[b]:cr[b + 1]].cpu(), w), b
        assert bool(torch.isnan(o._base[:, :, d:]).all())


def test_append_special_values(orbq):
    """Zeros, infinities, NaN, the smallest and largest numbers; a scale that was never written under
    a block's first token; a block that grows at every token."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    page, d, heads = 16, 64, 2
    c = cache_of(orbq, rng, 5, heads, d, page)
    c.k_scales.fill_(float("nan"))
    c.v_scales.fill_(float("nan"))
    x = rng.standard_normal((page, heads, d)).astype(np.float32)
    x[0] = 0.0
    x[1, 0, 3], x[1, 1, 4], x[2, 0, 5], x[3, 0, 0] = np.inf, -np.inf, np.nan, -0.0
    x[4] = 3.3e38
    x[5] = 1e-45
    want = host(c)
    table = np.array([[2], [4], [1]], np.int32)
    zero, far = np.zeros((3, heads, d), np.float32), np.full((2, heads, d), np.nan, np.float32)
    rows = np.concatenate([x, zero, far])
    cu = np.array([0, 16, 19, 21], np.int32)
    oa.kv_append(*want, table, [0, 0, 0], [x, zero, far], [x, zero, far])
    k = torch.from_numpy(rows).cuda()
    orbq.kv_append(c, k, k, ints(table), ints([0, 0, 0]), cu=ints(cu))
    compare_cache(c, want, table, [16, 3, 2], page)
    assert want[2][4, 0] == np.float32(2.0 ** -64)
    # one token at a time, each larger than the last: growth after growth
    c = cache_of(orbq, rng, 2, heads, d, page)
    want, table = host(c), np.array([[1]], np.int32)
    y = (rng.standard_normal((page, heads, d)) * 1.1 ** np.arange(page)[:, None, None]).astype(np.float32)
    yt = torch.from_numpy(y).cuda()
    for t in range(page):
        oa.kv_append(*want, table, [t], [y[t:t + 1]], [y[t:t + 1]])
        orbq.kv_append(c, yt[t:t + 1], yt[t:t + 1], ints(table), ints([t]))
        compare_cache(c, want, table, [t + 1], page)
    k, v = orbq.kv_read(c, ints(table), ints([0]), ints([0, page]), page, dtype=torch.float32)
    top = np.maximum(want[2][1], want[3][1])[None, :, None]
    assert np.all(np.abs(k.cpu().numpy() - y) <= 2.5 * top) and torch.isfinite(v).all()


def test_append_absent_blocks_and_bounds(orbq):
    """Blocks outside the table or the cache are dropped, not written anywhere; they read as zero."""
    torch = torch_mod()
    rng = np.random.default_rng(4)
    page, d, heads = 16, 64, 2
    c = cache_of(orbq, rng, 3, heads, d, page)
    want = host(c)
    table = np.array([[7, 1], [-1, 2147483647]], np.int32)      # three of the four are no blocks of this cache
    x, x64 = dev(rng.standard_normal((80, heads, d)))
    oa.kv_append(*want, table, [0, 0], [x64[:40].astype(np.float32), x64[40:].astype(np.float32)],
                 [x64[:40].astype(np.float32), x64[40:].astype(np.float32)])
    orbq.kv_append(c, x, x, ints(table), ints([0, 0]))
    for g, w in zip(host(c), want):
        assert np.array_equal(g, w)
    k, v = orbq.kv_read(c, ints(table), ints([0, 0]), None, 80, dtype=torch.float32)
    assert not k[:16].any() and not v[32:].any() and bool((k[16:32] != 0).any())
    # positions and counts that leave the arrays: nothing is touched outside them
    before = host(c)
    orbq.kv_append(c, x, x, ints(table), ints([-5, 2 ** 31 - 1]))
    orbq.kv_append(c, x, x, ints(table), ints([64, 64]), cu=ints([-3, 10 ** 9, -7]))
    for g, w in zip(host(c), before):
        assert np.array_equal(g, w)


# -------------------------------------------------------------------------------------- attention
def check_attention(o, lse, want, d, name, n_keys):
    o64, lse64, spread = want
    eps = 2.0 ** -11 + 2.0 ** -17 + 2 * (d + 8) * 2.0 ** -24 * spread[..., 1:2]
    tol = UNIT[name] * np.abs(o64) * (1 + eps) + eps * spread[..., 0:1] + n_keys * 2.0 ** -24 * spread[..., 2:3] + LEAST[name]
    err = np.abs(o.double().cpu().numpy() - o64)
    assert np.all(err <= tol), f"{np.nanmax(err / tol):.3g} of the tolerance"
    assert np.isfinite(o.double().cpu().numpy()).all()
    if lse is not None:
        g = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(g), np.isneginf(lse64))
        f = np.isfinite(lse64)
        assert np.all(np.abs(g - lse64)[f] <= 1e-5 + (d + 16) * 2.0 ** -23 * spread[..., 1][f] + 2.0 ** -22 * np.abs(lse64[f]))


def run_attention(orbq, name, d, page, heads, kv_heads, lens, new, block=0, window=0, scale=None, seed=0, peak=1.0,
                  vary=1.0, pads=None, max_len=None, absent=()):
    torch = torch_mod()
    rng = np.random.default_rng(seed + d + page + len(lens))
    pages = sum((n + page - 1) // page for n in lens) + 4
    table = table_of(rng, pages, lens, page, extra=2)
    c = cache_of(orbq, rng, pages, kv_heads, d, page)
    for s, w in ((c.k_scales, 1.0), (c.v_scales, vary)):
        s.copy_(torch.from_numpy((np.exp(w * rng.standard_normal((pages, kv_heads))) / 40).astype(np.float32)))
    held = sorted(set(int(x) for x in table.ravel() if x >= 0))
    nobody = [p for p in range(pages) if p not in held]
    c.k_scales[nobody] = float("nan")
    c.v_scales[nobody] = float("inf")
    for b, p in absent:
        table[b, p] = -1
    total = sum(new)
    cu = np.concatenate([[0], np.cumsum(new)])
    q, q64 = dev(rng.standard_normal((total, heads, d)) * peak, name)
    lse = torch.full((total, heads), 7.0, dtype=torch.float32, device="cuda")
    qq = strided(q, *pads) if pads else q
    out = strided(torch.zeros_like(q), *pads) if pads else None
    o = orbq.kv_attention(c, qq, ints(table), ints(lens), cu=ints(cu), max_new=max(new), causal_block=block, window=window,
                          scale=scale, lse=lse, out=out, max_len=max_len)
    kc, vc, ks, vs = host(c)
    sc = 1 / math.sqrt(d) if scale is None else scale
    for b, n in enumerate(lens):
        if not new[b]:
            continue
        k, v = oa.kv_tokens(kc, ks, table[b], n, False), oa.kv_tokens(vc, vs, table[b], n, True)
        want = oa.attention(q64[cu[b]:cu[b + 1]], k, v, block, window, sc)
        check_attention(o[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], want, d, name, n)
    if pads:
        assert bool(torch.isnan(o._base[:, :, d:]).all())
    return c, q, table, o


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 500, 1301]


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_one_query_token(orbq, name, d, page):
    for heads, kv_heads in ((4, 4), (8, 1), (14, 2), (34, 2)):     # 1, 8, 7 and 17 rows a cache head
        log(f"one token {name} d={d} page={page} heads {heads}/{kv_heads}")
        run_attention(orbq, name, d, page, heads, kv_heads, LENS, [1] * len(LENS), block=1, pads=(2, 8))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("block,window", [(0, 0), (1, 0), (1, 1), (1, 33), (0, 70), (7, 0), (50, 64), (300, 17)])
def test_masks(orbq, d, block, window):
    """Few and many rows, queries before the first token, sequences without queries, ragged lengths."""
    for heads, kv_heads, new in ((3, 3, [3, 1, 9, 2, 0, 5, 30, 4, 8, 17, 2]), (6, 2, [40, 1, 130, 20, 0, 64, 64, 65, 33, 200, 301])):
        log(f"masks d={d} block={block} window={window} heads {heads}/{kv_heads}")
        run_attention(orbq, "bf16" if d == 128 else "f16", d, 16 if d == 64 else 64, heads, kv_heads, LENS, new, block, window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_query_tokens(orbq, d):
    log(f"many d={d}")
    run_attention(orbq, "bf16", d, 128, 4, 4, [700, 129, 1000], [700, 128, 999], block=1, pads=(2, 8))
    run_attention(orbq, "f16", d, 32, 10, 2, [901, 300], [333, 300], block=100)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 70])
def test_scores_and_scales_of_every_size(orbq, d, new):
    """Sharp softmax, scales of blocks many orders apart, a negative, zero and large factor, far q."""
    log(f"sizes d={d} new={new}")
    for kw in (dict(peak=30.0), dict(vary=8.0), dict(scale=-0.2), dict(scale=0.0), dict(scale=1.5, peak=4.0),
               dict(peak=1e-6, scale=1e5), dict(peak=0.0)):
        run_attention(orbq, "bf16", d, 64, 4, 2, [1000, 77], [new, new], block=1, **kw)


def test_far_q_and_absent_blocks(orbq):
    run_attention(orbq, "bf16", 128, 64, 4, 2, [400], [2], scale=1e-32, peak=1e30)
    run_attention(orbq, "bf16", 128, 64, 4, 2, [400], [90], scale=1e32, peak=1e-30)
    for new in (1, 60):       # a block that the table does not have is not attended to
        run_attention(orbq, "bf16", 128, 16, 4, 2, [100, 300], [new, new], absent=((0, 0), (1, 5), (1, 18)))


@pytest.mark.parametrize("d,new,heads,kv_heads", [(64, 4, 16, 2), (128, 1, 8, 8), (256, 3, 4, 2), (128, 40, 2, 1)])
def test_long_cache_is_split_and_joined(orbq, d, new, heads, kv_heads):
    """One sequence over many workgroups, whatever the caller said about its length."""
    torch = torch_mod()
    log(f"long d={d}")
    c, q, table, o = run_attention(orbq, "f16", d, 128, heads, kv_heads, [20011], [new], block=1)
    for guess in (1, 300, 10 ** 6):
        o2 = orbq.kv_attention(c, q, ints(table), ints([20011]), causal_block=1, max_len=guess)
        assert (o2.float() - o.float()).abs().max().item() <= 2.0 ** -9 * o.float().abs().max().item()
    assert torch.equal(orbq.kv_attention(c, q, ints(table), ints([20011]), causal_block=1), o)   # no order of atomics


def test_not_finite_q_stays_in_its_row(orbq):
    torch = torch_mod()
    for new in (2, 80):
        c, q, table, o = run_attention(orbq, "bf16", 128, 64, 4, 2, [300], [new], block=1)
        q[0, 1, 5] = float("nan")
        q[1, 2, 7] = float("inf")
        o2 = orbq.kv_attention(c, q, ints(table), ints([300]), causal_block=1)
        assert bool(torch.isnan(o2[0, 1]).all())
        same = torch.ones(new, 4, dtype=torch.bool)
        same[0, 1] = same[1, 2] = False
        assert torch.equal(o2[same.cuda()], o[same.cuda()])


def test_offsets_past_32_bits(orbq):
    """Codes behind the first 2^31 bytes of a cache, written, read back and attended to."""
    torch = torch_mod()
    page, heads, d = 128, 8, 256
    pages = 2 ** 31 // (page * heads * d) + 9
    c = orbq.KVCache.create(pages, heads, d, page)
    rng = np.random.default_rng(6)
    table = ints([[pages - 1, 3, pages - 4]])
    n = 300
    k, k64 = dev(rng.standard_normal((n, heads, d)), "bf16")
    v, v64 = dev(rng.standard_normal((n, heads, d)), "bf16")
    orbq.kv_append(c, k, v, table, ints([0]))
    rk, rv = orbq.kv_read(c, table, ints([0]), None, n, dtype=torch.float32)
    assert (rk - k.float()).abs().max().item() <= 0.5001 * c.k_scales[table[0].long()].max().item()
    q, q64 = dev(rng.standard_normal((1, heads, d)), "bf16")
    q2, q264 = dev(rng.standard_normal((50, heads, d)), "bf16")
    for a, a64 in ((q, q64), (q2, q264)):
        o = orbq.kv_attention(c, a, table, ints([n]))
        want = oa.attention(a64, rk.double().cpu().numpy(), rv.double().cpu().numpy(), 0, 0, d ** -0.5)
        check_attention(o, None, want, d, "bf16", n)


def test_another_stream_and_graph(orbq):
    """Calls on a stream of their own, and a captured token step whose lengths change between replays."""
    torch = torch_mod()
    rng = np.random.default_rng(9)
    page, heads, d, batch = 16, 4, 64, 3
    r = orbq.Rope.create((24, 20, 20))
    lens0 = [5, 40, 64]
    c = cache_of(orbq, rng, 40, heads, d, page)
    table = ints(rng.permutation(40)[:36].reshape(batch, 12))
    start, lens = ints(lens0), ints([n + 1 for n in lens0])
    pos = torch.zeros((batch, 3), device="cuda")
    q, k, v = (dev(rng.standard_normal((batch, heads, d)), "bf16")[0] for _ in range(3))
    o = torch.empty_like(q)

    def step(cache, out):
        a, b = orbq.rope(r, pos, q, k)
        orbq.kv_append(cache, b, v, table, start)
        return orbq.kv_attention(cache, a, table, lens, causal_block=1, out=out)

    eager = orbq.KVCache(*(t.clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(c, o)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(step(eager, None), o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, o)
    for i in range(4):
        start += 1
        lens += 1
        pos.copy_(start[:, None].float().expand(-1, 3))
        for t in (q, k, v):
            t.copy_(dev(rng.standard_normal((batch, heads, d)), "bf16")[0])
        g.replay()
        want = step(eager, None)
        torch.cuda.synchronize()
        assert torch.equal(o, want), i
        for x, y in zip(host(c)[2:], host(eager)[2:]):
            assert np.array_equal(x, y)


def test_refusals_of_the_binding(orbq):
    torch = torch_mod()
    c = orbq.KVCache.create(4, 2, 64, 16)
    table, one = ints([[0, 1]]), ints([3])
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    ok = lambda: orbq.kv_attention(c, x, table, ints([3]))  # noqa: E731
    ok()
    bad = [
        lambda: orbq.kv_attention(c, x.float(), table, one), lambda: orbq.kv_attention(c, x[:, :1], table, one),
        lambda: orbq.kv_attention(c, x[:, :, :32], table, one), lambda: orbq.kv_attention(c, x, table.long(), one),
        lambda: orbq.kv_attention(c, x, table, ints([3, 4])), lambda: orbq.kv_attention(c, x.cpu(), table, one),
        lambda: orbq.kv_attention(c, x, table, one, scale=float("nan")),
        lambda: orbq.kv_attention(c, x, table, one, window=-1), lambda: orbq.kv_attention(c, x, table, one, cu=ints([0])),
        lambda: orbq.kv_attention(c, x, table, one, out=x.float()),
        lambda: orbq.kv_attention(c, x, table, one, lse=torch.zeros(2, 3, device="cuda")),
        lambda: orbq.kv_append(c, x, x[:1], table, one), lambda: orbq.kv_append(c, x, x.half(), table, one),
        lambda: orbq.kv_append(c, x, x, table, ints([3, 3])),
        lambda: orbq.kv_append(orbq.KVCache(c.k_codes, c.v_codes[:3], c.k_scales, c.v_scales), x, x, table, one),
        lambda: orbq.kv_append(orbq.KVCache(c.k_codes.float(), c.v_codes, c.k_scales, c.v_scales), x, x, table, one),
        lambda: orbq.kv_read(c, table, one, None, 2, out=(x[:1], x[:1])),
        lambda: orbq.rope(orbq.Rope.create((64, 2)), torch.zeros((2, 2), device="cuda"), x),
        lambda: orbq.rope(orbq.Rope.create((32,)), torch.zeros((2, 2), device="cuda"), x),
        lambda: orbq.rope(orbq.Rope.create((32,), layout="odd"), torch.zeros((2, 1), device="cuda"), x),
        lambda: orbq.rope(orbq.Rope.create((32,)), torch.zeros((3, 1), device="cuda"), x),
        lambda: orbq.rope(orbq.Rope.create((32,)), torch.zeros((2, 1), device="cuda"), x, x.half()),
        lambda: orbq.rope(orbq.Rope.create((32,)), torch.zeros((2, 1), device="cuda"), x.transpose(1, 2)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(orbq.OrbqError):
            f()
            log(f"call {i} was not refused")
    # a workspace too small for a split call
    big = orbq.KVCache.create(600, 1, 64, 128)
    t = ints(np.arange(600)[None])
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    need = orbq.kv_attention_workspace_bytes(big, 1, 1, 1, 1, 600 * 128)
    assert need > 0
    with pytest.raises(orbq.OrbqError) as e:
        orbq.kv_attention(big, q, t, ints([0]), workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
    o = orbq.kv_attention(big, q, t, ints([0]), workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert not o.any()


@pytest.mark.parametrize("d,heads,kv_heads,lens,new,kw", [
    (128, 4, 4, [1500, 1100], [1030, 1100], dict(block=1)),
    (128, 6, 2, [700, 900], [400, 900], dict(block=37, window=130, absent=((0, 3), (1, 0), (1, 9)))),
    (256, 2, 1, [800, 5], [300, 600], dict(block=0, absent=((0, 12),))),
    (256, 1, 1, [9000], [700], dict(block=1)),
    (128, 2, 2, [9000], [1200], dict(block=300, window=2000))])
def test_many_rows_with_tiles_turned_before_or_on_the_way(orbq, d, heads, kv_heads, lens, new, kw):
    """Enough rows that the tiles are laid out in the workspace first; a guess at the lengths below what the
    table holds forbids that, and gives the same up to rounding."""
    log(f"turned d={d} lens={lens} new={new} {kw}")
    kw = dict(kw)
    block, window = kw.get("block", 0), kw.get("window", 0)
    c, q, table, o = run_attention(orbq, "bf16", d, 64, heads, kv_heads, lens, new, **kw)
    cu = ints(np.concatenate([[0], np.cumsum(new)]))
    args = dict(cu=cu, max_new=max(new), causal_block=block, window=window)
    full = table.shape[1] * 64
    assert orbq.kv_attention_workspace_bytes(c, len(lens), sum(new), max(new), heads, full, block, window) >= \
        len(lens) * kv_heads * 64 * 4 * d                       # the f16 tiles are there
    o2 = orbq.kv_attention(c, q, ints(table), ints(lens), max_len=max(lens) // 2, **args)
    assert (o2.float() - o.float()).abs().max().item() <= 2.0 ** -7 * o.float().abs().max().item()


@pytest.mark.parametrize("d,heads,kv_heads,lens,new,window,turned", [
    (64, 8, 2, [777], [1], 35, False), (128, 4, 4, [777], [1], 35, False), (256, 4, 2, [777], [1], 35, False),
    (128, 48, 4, [900], [3], 35, False), (64, 4, 2, [900], [90], 90, False), (128, 4, 2, [900], [90], 90, False),
    (256, 4, 2, [900], [90], 90, False), (128, 2, 2, [4600], [2100], 1900, True), (256, 1, 1, [2600], [1500], 1000, True)])
def test_blocks_before_the_window_may_hold_anything(orbq, d, heads, kv_heads, lens, new, window, turned):
    """Pages that no query of the call sees, in the tile where the first window begins among them, hold scales that are
    no numbers."""
    torch = torch_mod()
    log(f"before the window d={d} new={new}")
    page = 16
    first = lens[0] - new[0] + 1 - window            # the first visible token
    assert first > 16 and first % 64 >= 16           # and there is a block before it in its tile
    c, q, table, o = run_attention(orbq, "bf16", d, page, heads, kv_heads, lens, new, block=1, window=window)
    tiles = orbq.kv_attention_workspace_bytes(c, 1, new[0], new[0], heads, table.shape[1] * page, 1, window)
    assert (tiles >= kv_heads * (window + new[0]) * 4 * d) == turned
    hidden = torch.from_numpy(table[0, :first // page].astype(np.int64)).cuda()
    for k, v in (("inf", "inf"), ("-inf", "nan"), ("nan", "-inf")):
        c.k_scales[hidden] = float(k)
        c.v_scales[hidden] = float(v)
        assert torch.equal(orbq.kv_attention(c, q, ints(table), ints(lens), causal_block=1, window=window), o), (k, v)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 70])
def test_scores_of_the_largest_magnitude(orbq, d, new):
    """Scores down to -2^25: the largest takes all the weight, as with small ones."""
    torch = torch_mod()
    page, heads, n = 64, 2, 300
    c = orbq.KVCache.create(8, heads, d, page)
    rng = np.random.default_rng(d + new)
    table = ints(np.arange(5)[None])
    k = np.zeros((n, heads, d), np.float32)
    k[:, :, 0] = -rng.uniform(90, 127, (n, 1))
    v = rng.standard_normal((n, heads, d)).astype(np.float32)
    orbq.kv_append(c, dev(k)[0], dev(v)[0], table, ints([0]))
    rk, rv = orbq.kv_read(c, table, ints([0]), None, n, dtype=torch.float32)
    q = torch.zeros((new, heads, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0 ** 18                                    # times 127: just below 2^25
    lse = torch.empty((new, heads), device="cuda")
    o = orbq.kv_attention(c, q, table, ints([n]), lse=lse, scale=1.0)
    for h in range(heads):
        top = rk[:, h, 0].max()
        assert bool((rk[rk[:, h, 0] != top, h, 0] < top * 1.00001).all())   # the next is far behind
        mean = rv[rk[:, h, 0] == top, h].double().mean(0)     # equal keys share the weight
        err = (o[:, h].double() - mean).abs()
        assert bool((err <= 2.0 ** -8 * mean.abs() + 2.0 ** -10 * rv.abs().max()).all())
        want = top.double() * 2.0 ** 18
        assert -2.0 ** 25 < rk[:, h, 0].min().item() * 2.0 ** 18 < -2.0 ** 24.9 and bool(((lse[:, h].double() - want) / want).abs().max() <= 1e-6)


def test_a_table_without_pages(orbq):
    """Nothing is held: appending writes nothing, reading gives zeros, attention sees nothing."""
    torch = torch_mod()
    c = orbq.KVCache.create(2, 2, 64, 16)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.fill_(3)
    table = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    for each in (1, 70):
        x = torch.ones((2 * each, 2, 64), dtype=torch.bfloat16, device="cuda")
        orbq.kv_append(c, x, x, table, ints([0, 5]))
        assert all(bool((t == 3).all()) for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales))
        k, v = orbq.kv_read(c, table, ints([0, 5]), None, 2 * each)
        assert not k.any() and not v.any()
        lse = torch.zeros((2 * each, 2), device="cuda")
        assert not orbq.kv_attention(c, x, table, ints([0, 9]), lse=lse).any()
        assert bool(torch.isneginf(lse).all())


def test_a_workspace_elsewhere_is_refused(orbq):
    torch = torch_mod()
    c = orbq.KVCache.create(600, 1, 64, 128)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(orbq.OrbqError) as e:
            orbq.kv_attention(c, q, ints(np.arange(600)[None]), ints([0]), workspace=ws)
        assert e.value.status == -1


@pytest.mark.parametrize("d,heads,kv_heads,lens,new,block,window", [
    (128, 53, 53, [1500, 3, 800, 0, 1333], 100, 0, 0), (128, 53, 53, [1500, 3, 800, 100, 1333], 100, 1, 0),
    (256, 262, 131, [700], 100, 30, 0), (256, 262, 131, [700], 100, 0, 400), (64, 390, 390, [600, 511], 70, 1, 0)])
def test_only_the_last_round_of_row_tiles_is_split(orbq, d, heads, kv_heads, lens, new, block, window):
    """Some row tiles more than fill the card once: those alone are split and joined."""
    log(f"last round d={d} heads {heads}/{kv_heads} {lens} {block} {window}")
    c, q, table, o = run_attention(orbq, "bf16", d, 64, heads, kv_heads, lens, [new] * len(lens), block, window)
    n = orbq.kv_attention_workspace_bytes(c, len(lens), len(lens) * new, new, heads, table.shape[1] * 64, block, window)
    assert 0 < n < len(lens) * new * heads * 2 * (d + 2) * 4       # less than two parts of every row
    assert torch_mod().equal(orbq.kv_attention(c, q, ints(table), ints(lens), causal_block=block, window=window), o)


@pytest.mark.parametrize("d,most", [(64, 2), (128, 2), (256, 2), (128, 80)])
def test_rows_beyond_the_bound_are_left_alone(orbq, d, most):
    """Rows of a sequence past max_new, and rows of no sequence, are not written, split keys or not."""
    torch = torch_mod()
    rng = np.random.default_rng(d)
    for n in (200, 30000):
        pages = -(-n // 128)
        c = cache_of(orbq, rng, pages, 2, d, 128)
        q, _ = dev(rng.standard_normal((most + 9, 2, d)), "bf16")
        out, lse = torch.full_like(q, 7.0), torch.full((most + 9, 2), 7.0, device="cuda")
        orbq.kv_attention(c, q, ints(np.arange(pages)[None]), ints([n]), cu=ints([0, most + 5]), max_new=most, out=out, lse=lse)
        assert bool((out[most:] == 7.0).all()) and bool((lse[most:] == 7.0).all())
        assert bool((out[:most] != 7.0).any(-1).all()) and bool((lse[:most] != 7.0).all())
