"""kv_append_rope on the GPU.  Without norms it is held, bit for bit, to rope and kv_append of the same values in 32 bits
(which have the float64 oracle's tests); with them, to the definition in 64 bits.

Tolerances of the normalised case, from the arithmetic before any run, e = 2^-24: the sum of a head's squares is taken in 8 + 5
steps, so the factor 1 / sqrt(..) is off by at most 10 e relative, the products with it and the weight by 2 e more, the turn by
5e-7 (|a| + |b|) of its pair (tests/test_gpu_attention.py): together 13 e + 5e-7 < 1.3e-6 of |a| + |b|.  A code is then the nearest
to its value within 0.5 + 127 1.3e-6 2 steps, a fresh page's scale within 1.3e-6 2 relative."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_common import log, torch_mod

pytestmark = pytest.mark.gpu
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
REL = 1.3e-6


@pytest.fixture(scope="module")
def orbq():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import calibration_free_w4a4_amd as m
    m.load()
    return m


def ints(v):
    return torch_mod().tensor(np.asarray(v), dtype=torch_mod().int32, device="cuda")


class Case:
    def __init__(self, orbq, new, held, qh, kh, d, page, dims, layout, name, seed=0):
        torch = torch_mod()
        self.orbq, self.new, self.held, self.name = orbq, new, held, name
        self.dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        total = sum(new)
        x = (normal(total, qh + 2 * kh, d) * torch.exp(0.5 * normal(total, qh + 2 * kh, 1))).to(self.dtype)
        self.q, self.k, self.v = x[:, :qh], x[:, qh:qh + kh], x[:, qh + kh:]       # parts of one tensor
        lens = [a + b for a, b in zip(held, new)]
        per = [(n + page - 1) // page for n in lens]
        order = torch.randperm(sum(per) + 2, generator=torch.Generator().manual_seed(seed))
        self.table = torch.full((len(new), max(per) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        self.table = self.table.cuda()
        self.kc = torch.randint(-127, 128, (sum(per) + 2, kh, page, d), generator=gen, device="cuda").to(torch.int8)
        self.vc = torch.randint(-127, 128, (sum(per) + 2, kh, d, page), generator=gen, device="cuda").to(torch.int8)
        self.ks, self.vs = (torch.exp(normal(sum(per) + 2, kh)) / 60 for _ in range(2))
        self.rope = orbq.Rope.create(dims, layout=layout)
        self.pos = torch.floor(normal(total, len(dims)).abs() * 500)
        self.w = 1 + 0.2 * normal(2, d)
        self.start, self.cu = ints(held), ints(np.concatenate([[0], np.cumsum(new)]))

    def cache(self):
        return self.orbq.KVCache(self.kc.clone(), self.vc.clone(), self.ks.clone(), self.vs.clone())

    def call(self, cache, **kw):
        f = dict(cache=cache, rope=self.rope, positions=self.pos, q=self.q, k=self.k, v=self.v, table=self.table, start=self.start,
                 cu=self.cu, max_new=max(self.new))
        f.update(kw)
        return self.orbq.kv_append_rope(**f)

    def apart(self, cache):
        """q' and the cache by rope and kv_append in 32 bits."""
        q, k = self.orbq.rope(self.rope, self.pos, self.q.float(), self.k.float())
        self.orbq.kv_append(cache, k, self.v.float(), self.table, self.start, cu=self.cu, max_new=max(self.new))
        return q.to(self.dtype)


def same(a, b):
    torch = torch_mod()
    return all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("k_codes", "v_codes", "k_scales", "v_scales"))


CASES = [
    # new, held, q heads, kv heads, d, page, dims, layout
    ([1], [0], 1, 1, 64, 16, (64,), "pairs"), ([1], [77], 12, 12, 128, 64, (44, 42, 42), "pairs"),
    ([1] * 9, [5, 0, 63, 64, 65, 127, 300, 16, 31], 32, 8, 128, 64, (128,), "halves"),
    ([70, 1, 33], [3, 200, 0], 6, 3, 64, 32, (16, 24, 24), "halves"), ([130, 257], [0, 100], 4, 2, 256, 128, (64, 64, 64), "pairs"),
    ([5, 0, 17, 2], [1, 2, 3, 4], 4, 4, 64, 16, (32,), "halves"), ([40, 3], [9, 12], 2, 1, 128, 16, (30, 6), "pairs"),
    ([40, 3], [9, 12], 2, 1, 128, 32, (30, 6), "halves"), ([17], [15], 3, 3, 256, 16, (256,), "halves"),
    ([200], [1000], 8, 1, 64, 128, (20, 20, 20, 4), "pairs"), ([300, 11, 129], [0, 64, 1], 24, 8, 128, 128, (16, 56, 56), "halves"),
    ([1000], [28], 2, 2, 256, 64, (100,), "halves"), ([640, 640], [0, 0], 40, 4, 64, 64, (2,), "halves")]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new,held,qh,kh,d,page,dims,layout", CASES)
def test_is_rope_and_append(orbq, new, held, qh, kh, d, page, dims, layout, name):
    log(f"kv_append_rope {name} new={new} held={held} heads {qh}/{kh} d={d} page={page} {dims} {layout}")
    torch = torch_mod()
    c = Case(orbq, new, held, qh, kh, d, page, dims, layout, name)
    want, got = c.cache(), c.cache()
    q_want, q = c.apart(want), c.call(got)
    assert torch.equal(q, q_want) and same(got, want)
    # again, q in place: nothing depends on what was there but the cache
    third = c.cache()
    x = c.q.clone()
    assert c.call(third, q=x, out=x) is x
    assert torch.equal(x, q_want) and same(third, want)
    wide = torch.full((x.shape[0], qh + 2, d + 16), 9.0, dtype=c.dtype, device="cuda")
    c.call(c.cache(), out=wide[:, 1:qh + 1, :d])
    assert torch.equal(wide[:, 1:qh + 1, :d], q_want) and bool((wide[:, :, d:] == 9).all()) and bool((wide[:, [0, -1]] == 9).all())


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new,held,qh,kh,d,page,dims,layout", CASES)
def test_with_norms(orbq, new, held, qh, kh, d, page, dims, layout, name):
    log(f"kv_append_rope, norms {name} new={new} held={held} heads {qh}/{kh} d={d} page={page} {dims} {layout}")
    torch = torch_mod()
    c = Case(orbq, new, held, qh, kh, d, page, dims, layout, name, seed=1)
    eps = 1e-3
    cache, plain = c.cache(), c.cache()
    q = c.call(cache, q_weight=c.w[0], k_weight=c.w[1], eps=eps)
    c.apart(plain)
    assert torch.equal(cache.v_codes, plain.v_codes) and torch.equal(cache.v_scales, plain.v_scales)
    turned = []
    for x, w in ((c.q, c.w[0]), (c.k, c.w[1])):
        x = x.double().cpu().numpy()
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
        y = oa.rope(x, c.rope.dims, c.rope.freqs.cpu().numpy(), c.pos.cpu().numpy(), layout)
        a, b = oa.rope_pairs(c.rope.dims, layout)
        size = np.abs(x)
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        turned.append((y, size))
    (q64, size), (k64, _) = turned
    err = np.abs(q.double().cpu().numpy() - q64)
    assert np.all(err <= REL * size + UNIT[name] * np.abs(q64) * (1 + 1e-5) + 2.0 ** -24)
    # keys, page by page: every new one has its nearest code; what the page held is as the rule says
    kc, ks, table = cache.k_codes.cpu().numpy().astype(np.int64), cache.k_scales.double().cpu().numpy(), c.table.cpu().numpy()
    kc0, ks0 = c.kc.cpu().numpy().astype(np.float64), c.ks.double().cpu().numpy()
    untouched = set(range(len(ks)))
    row = 0
    for b, (n, h) in enumerate(zip(new, held)):
        for p in range(h // page, (h + n + page - 1) // page) if n else ():
            lo, hi = max(h, p * page), min(h + n, (p + 1) * page)
            x, pg, had = k64[row + lo - h:row + hi - h].transpose(1, 0, 2), table[b, p], lo - p * page
            untouched.discard(pg)
            need = np.maximum(np.abs(x).max((1, 2)) / 127, 2.0 ** -64)
            s = ks[pg]
            for head in range(kh):
                if had == 0:
                    assert abs(s[head] / need[head] - 1) <= 2 * REL
                elif need[head] <= ks0[pg, head] * (1 - 2 * REL):
                    assert s[head] == ks0[pg, head]
                elif need[head] > ks0[pg, head] * (1 + 2 * REL):
                    assert abs(s[head] / max(need[head], 1.25 * ks0[pg, head]) - 1) <= 2 * REL
                off = np.abs(x[head] / s[head] - kc[pg, head, had:had + hi - lo])
                assert np.all(off <= 0.5 + 127 * 2 * REL)
                if had:
                    off = np.abs(kc0[pg, head, :had] * (ks0[pg, head] / s[head]) - kc[pg, head, :had])
                    assert np.all(off <= 0.5 + 127 * 2 * REL)
        row += n
    rest = sorted(untouched)
    assert torch.equal(cache.k_codes[rest], c.kc[rest]) and torch.equal(cache.k_scales[rest], c.ks[rest])
    # one norm alone
    one = c.call(c.cache(), q_weight=c.w[0], eps=eps)
    assert torch.equal(one, q)
    other = c.cache()
    assert torch.equal(c.call(other, k_weight=c.w[1], eps=eps), c.apart(c.cache())) and same(other, cache)


def test_bounds_absent_pages_and_shared_positions(orbq):
    torch = torch_mod()
    c = Case(orbq, [20, 30, 40, 6], [10, 3, 0, 50], 4, 2, 64, 16, (64,), "halves", "bf16")
    # a page that is absent, one outside the cache, a sequence that does not begin yet: their keys go nowhere, q is turned
    c.table[0, 1], c.table[1, 0] = -1, 10 ** 6
    c.start[3] = -5
    want, got = c.cache(), c.cache()
    q_want, q = c.apart(want), c.call(got)
    assert torch.equal(q, q_want) and same(got, want)
    # no pages at all
    q = c.call(got, table=c.table[:, :0])
    assert torch.equal(q, q_want) and same(got, want)
    # without q; rows behind the last sequence, and beyond the bound, are left alone
    got = c.cache()
    assert c.call(got, q=None) is None and same(got, want)
    c.cu.copy_(ints([2, 20, 20, 60, 70]))
    want, got = c.cache(), c.cache()
    out = torch.full_like(c.q, 5.0, memory_format=torch.contiguous_format)
    q_want, _ = orbq.rope(c.rope, c.pos, c.q, c.k)
    c.call(got, max_new=17, out=out)
    done = torch.zeros(96, dtype=torch.bool)
    for a, b in ((2, 20), (20, 60), (60, 70)):
        done[a:min(b, a + 17)] = True
    assert torch.equal(out[done], q_want[done]) and bool((out[~done] == 5).all())
    k = orbq.rope(c.rope, c.pos, c.k.float())
    orbq.kv_append(want, k, c.v.float(), c.table, c.start, cu=c.cu, max_new=17)
    assert same(got, want)
    # a batch of equal sequences shares one set of positions
    c = Case(orbq, [12, 12, 12], [0, 16, 5], 2, 2, 64, 16, (20, 12), "pairs", "f16")
    shared = c.pos[:12].contiguous()
    c.pos = shared.repeat(3, 1)
    a, b = c.cache(), c.cache()
    assert torch.equal(c.call(a), c.call(b, positions=shared, cu=None, max_new=None)) and same(a, b)


def test_special_values(orbq):
    """A NaN or an infinity among k loses its pair and, with a norm, its head's row; zero rows stay zero."""
    torch = torch_mod()
    c = Case(orbq, [16], [0], 2, 2, 64, 16, (32,), "pairs", "f32")
    q, k = c.q.clone(), c.k.clone()
    q[3], k[3] = 0, 0
    k[5, 0, 4], k[6, 1, 40], q[7, 1, 9] = float("nan"), float("inf"), -float("inf")
    want, got = c.cache(), c.cache()
    qw, kw = orbq.rope(c.rope, c.pos, q, k)
    orbq.kv_append(want, kw, c.v, c.table, c.start, cu=c.cu)
    out = c.call(got, q=q, k=k)
    assert torch.equal(out.nan_to_num(7), qw.nan_to_num(7)) and same(got, want)
    got = c.cache()
    out = c.call(got, q=q, k=k, q_weight=c.w[0], k_weight=c.w[1])
    codes = got.k_codes[c.table[0, 0]]
    assert not out[3].any() and not codes[:, 3].any() and bool((codes[0, 5] == 0).all()) and bool(torch.isfinite(got.k_scales[c.table[0, 0]]).all())
    assert bool(torch.isfinite(out[[i for i in range(16) if i != 7]]).all()) and bool(torch.isfinite(out[7, 0]).all())


def test_graph_and_streams(orbq):
    """A captured step follows the device's counts and positions."""
    torch = torch_mod()
    c = Case(orbq, [1] * 5, [3, 15, 16, 40, 0], 8, 2, 128, 16, (44, 42, 42), "pairs", "bf16")
    table = torch.arange(5 * 8, dtype=torch.int32, device="cuda").view(5, 8)
    kc, vc = torch.zeros((40, 2, 16, 128), dtype=torch.int8, device="cuda"), torch.zeros((40, 2, 128, 16), dtype=torch.int8, device="cuda")
    pair = [orbq.KVCache(kc.clone(), vc.clone(), torch.ones(40, 2, device="cuda"), torch.ones(40, 2, device="cuda")) for _ in range(2)]
    start, x = c.start.clone(), [t.contiguous() for t in (c.q, c.k, c.v)]
    call = lambda cache, s: orbq.kv_append_rope(cache, c.rope, c.pos, *x, table, s, q_weight=c.w[0], k_weight=c.w[1])  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(orbq.KVCache(kc.clone(), vc.clone(), torch.ones(40, 2, device="cuda"), torch.ones(40, 2, device="cuda")), start)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call(pair[0], start)
        start += 1
    start.copy_(c.start)
    mine = c.start.clone()
    for k in range(4):
        for t in x:
            t.mul_(1.3)
        c.pos.add_(1)
        graph.replay()
        want = call(pair[1], mine)
        mine += 1
        torch.cuda.synchronize()
        assert torch.equal(q, want) and same(*pair) and torch.equal(start, mine)


def test_refusals(orbq):
    torch = torch_mod()
    c = Case(orbq, [4, 4], [0, 0], 4, 2, 64, 16, (32,), "pairs", "bf16")
    w = c.w[0].contiguous()
    bad = [dict(q=c.q.float()), dict(q=c.q[:5]), dict(q=c.q[..., :32]), dict(k=c.k[:, :1]), dict(v=c.v.half()), dict(k=c.k.cpu()),
           dict(positions=c.pos[:3]), dict(positions=c.pos.double()), dict(positions=c.pos[:, :0]), dict(start=c.start.long()),
           dict(start=c.start[:1]), dict(cu=c.cu[:2]), dict(table=c.table.long()), dict(q_weight=w.bfloat16()), dict(k_weight=w[:32]),
           dict(q=None, q_weight=w), dict(out=c.q.float()), dict(out=c.q[:2]), dict(eps=-1.0), dict(eps=float("nan")),
           dict(q=c.q[..., 1:]), dict(rope=orbq.Rope.create((128,))), dict(max_new=-1),
           dict(out=torch.empty((8, 1, 64), dtype=torch.bfloat16, device="cuda").expand(8, 4, 64))]
    for kw in bad:
        with pytest.raises(orbq.OrbqError):
            c.call(c.cache(), **kw)
    leaf = c.q.clone().requires_grad_()
    q = c.call(c.cache(), q=leaf)
    with pytest.raises(orbq.OrbqError):
        q.float().sum().backward()
    with torch.no_grad():
        assert not c.call(c.cache(), q=leaf).requires_grad


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_every_form(orbq, name, d, layout):
    """Every page size, whole and part of the head turned, in whole columns of 8 and not, a token and several pages: the bits of rope
    and kv_append without norms, and with norms whose weights are 1 of rows that are normalised to a power of two already."""
    torch = torch_mod()
    ones = torch.ones(d, device="cuda")
    for page in (16, 32, 64, 128):
        for dims in ((d,), (d // 2,), (d // 4, 6)):
            for new in ([1, 1], [2 * page + 5, 3]):
                c = Case(orbq, new, [3, page - 1], 5, 3, d, page, dims, layout, name, seed=page + d)
                want, got = c.cache(), c.cache()
                q_want, q = c.apart(want), c.call(got)
                assert torch.equal(q, q_want) and same(got, want), (page, dims, new)
                # entries of magnitude 2: the mean square is 4, its root 2, exactly, and so is the quotient
                c.q, c.k = (torch.where(t > 0, 2.0, -2.0).to(c.dtype) for t in (c.q, c.k))
                got, half = c.cache(), c.cache()
                q = c.call(got, q_weight=ones, k_weight=ones, eps=0.0)
                c.q, c.k = c.q / 2, c.k / 2
                assert torch.equal(q, c.apart(half)) and same(got, half), (page, dims, new)
