"""The products with bias, activation, gate and residual on the GPU, against float64 (oracle.epilogue of the exact product of the
decoded bf16 centroids).

Tolerances, from the arithmetic before any run, e = 2^-24:
  * products of bf16 are exact in fp32; they are added 16 or 32 at a time, d / 16 times, each sum off by 2 e of its size at most, and
    the splits of the few-row form by 16 e more: (d / 8 + 32) e of sum |a| |b| s r, with the two scales' products 4 e more;
  * bias: 2 e of both;  GELU: its slope is below 1.13, its own arithmetic (exp2 and the reciprocal to an ulp, Phi to 1.5e-7) below
    6e-7 |x|;  gate and residual: 2 e of each;  half a step of the output's type (2^-8 or 2^-24).
"""
import numpy as np
import pytest

import oracle
import workloads
from oracle.block_norm import groups_of
from oracle.epilogue import epilogue
from tests.conftest import oracle_codebook
from tests.gpu_common import dense_pi, dev_bf16, log, torch_mod

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


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
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def dev(x, name):
    t = torch_mod().from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype_of(name)).cuda()
    return t, t.double().cpu().numpy()


class Case:
    """Random codes, scales and epilogue vectors; the exact product and the size of its terms."""

    def __init__(self, orbq, n, m, d, ba, bw, groups=1, cu=None, vectors="bf16", seed=0, x=True):
        rng = np.random.default_rng([seed, n, m, d, ba])
        torch = torch_mod()
        self.orbq, self.n, self.m, self.d, self.groups, self.cu = orbq, n, m, d, groups, cu
        self.cb_w = orbq.Codebook.from_centroids(d, bw, oracle_codebook(d, bw))
        kw = rng.integers(0, 1 << bw, (m, d))
        self.w = torch.from_numpy(oracle.pack_codes(kw, bw)).cuda(), dev_bf16(workloads.bf16_bits_from_f64(rng.uniform(1, 4, m)))
        b = oracle.decode_lut_bf16(oracle_codebook(d, bw))[kw] * self.w[1].double().cpu().numpy()[:, None]
        self.b = b
        if x:
            self.cb_a = orbq.Codebook.from_centroids(d, ba, oracle_codebook(d, ba))
            kx = rng.integers(0, 1 << ba, (n, d))
            s = torch.from_numpy((np.sqrt(d) * rng.uniform(0.2, 1.0, n)).astype(np.float32)).cuda()
            self.x = torch.from_numpy(oracle.pack_codes(kx, ba)).cuda(), s
            a = oracle.decode_lut_bf16(oracle_codebook(d, ba))[kx] * s.double().cpu().numpy()[:, None]
            self.product, self.size = a @ b.T, np.abs(a) @ np.abs(b).T
        self.t, self.v = {}, {}
        for name, shape, kind in (("bias", (m,), vectors), ("gate", (groups, m), vectors)):
            self.t[name], self.v[name] = dev(rng.standard_normal(shape), kind)
        self.t["residual"], self.v["residual"] = {}, {}
        for kind in ("f32", "bf16"):
            self.t["residual"][kind], self.v["residual"][kind] = dev(3 * rng.standard_normal((n, m)), kind)

    def how(self, parts, name):
        out = {a: self.t[a] for a in ("bias", "gate") if a in parts}
        if "residual" in parts:
            out["residual"] = self.t["residual"][name]
        if self.cu is not None:
            out["cu"] = torch_mod().tensor(self.cu, dtype=torch_mod().int32, device="cuda")
        return out

    def call(self, parts, act, name, **kw):
        return self.orbq.lut_gemm(*self.x, self.cb_a, *self.w, self.cb_w, self.d, out_dtype=dtype_of(name), act=act,
                                  **self.how(parts, name), **kw)

    def check(self, got, parts, act, name, product=None, size=None, rel=None):
        product = self.product if product is None else product
        size = self.size if size is None else size
        v = {a: (self.v[a] if a in parts else None) for a in ("bias", "gate")}
        v["residual"] = self.v["residual"][name] if "residual" in parts else None
        want = epilogue(product, act, v["bias"], v["gate"], v["residual"], self.groups, self.cu)
        rows = [i for g in groups_of(self.n, self.groups, self.cu) for i in g]
        pre = product + (0 if v["bias"] is None else v["bias"])
        tol = ((self.d / 8 + 36) * E if rel is None else rel) * size + (0 if v["bias"] is None else 2 * E * (np.abs(v["bias"]) + np.abs(pre)))
        if act != "none":
            tol = 1.13 * tol + 6e-7 * np.abs(pre)
        if v["gate"] is not None:
            for g, at in enumerate(groups_of(self.n, self.groups, self.cu)):
                tol[list(at)] *= np.abs(v["gate"][g if len(v["gate"]) > 1 else 0])
        tol += 2 * E * (np.abs(want) + (0 if v["residual"] is None else 2 * np.abs(v["residual"]))) + UNIT[name] * np.abs(want) * (1 + 1e-5)
        err = np.abs(got.double().cpu().numpy() - want)[rows]
        assert np.all(err <= tol[rows]), f"{(err / tol[rows]).max():.3g} of the tolerance, {np.sum(err > tol[rows])} of {err.size}"


ALL = ("bias", "gate", "residual")
SHAPES = [
    # n, m, d, activation and weight bits, groups, cu: few rows ...
    (1, 8, 128, 4, 4, 1, None), (5, 200, 256, 4, 4, 5, None), (16, 1000, 1536, 4, 2, 2, None), (17, 264, 384, 3, 3, 3, [0, 5, 5, 17]),
    (31, 4104, 256, 2, 2, 1, None), (40, 88, 640, 6, 4, 4, None), (64, 5000, 256, 4, 6, 3, [2, 10, 40, 60]), (33, 136, 2176, 2, 4, 1, None),
    (7, 72, 256, 2, 6, 7, None), (64, 40, 4096, 6, 2, 2, None), (3, 24, 512, 6, 6, 1, None),
    # ... and tiles: whole, ragged, with an odd count of K tiles, of either shape
    (65, 200, 256, 4, 4, 5, None), (16, 72, 320, 4, 4, 2, None), (384, 192, 256, 4, 4, 1, None), (512, 256, 192, 2, 4, 2, None),
    (300, 520, 448, 3, 3, 3, [0, 100, 100, 300]), (1000, 760, 256, 6, 4, 4, [7, 300, 500, 700, 990]), (400, 1000, 128, 4, 2, 400, None),
    (700, 264, 576, 6, 6, 2, None), (257, 8, 64, 4, 6, 1, None), (2000, 1536, 192, 2, 2, 3, [0, 900, 1900, 2000])]


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,d,ba,bw,groups,cu", SHAPES)
def test_lut_gemm(orbq, n, m, d, ba, bw, groups, cu, name):
    log(f"lut_gemm fused {name} n={n} m={m} d={d} A{ba} W{bw} groups={groups} cu={cu}")
    c = Case(orbq, n, m, d, ba, bw, groups, cu, vectors="f32" if n % 2 else "bf16")
    for parts, act in ((ALL, "none"), (("bias",), "gelu_tanh"), (("gate", "residual"), "gelu_erf"), (("residual",), "none"),
                       (("bias", "gate"), "none")):
        c.check(c.call(parts, act, name), parts, act, name)
    # one gate for all rows
    if cu is None:
        c.t["gate"], c.v["gate"], c.groups = c.t["gate"][0], c.v["gate"][:1], 1
        c.check(c.call(ALL, "none", name), ALL, "none", name)


@pytest.mark.parametrize("ba,bw", [(2, 2), (2, 4), (2, 6), (3, 3), (4, 2), (4, 4), (4, 6), (6, 2), (6, 4), (6, 6)])
def test_every_few_row_form(orbq, ba, bw):
    """16, 32 and 64 tokens of a workgroup, 16 and 32 weight rows, 16 and 4 waves; one and several super-steps of a wave, ends within
    a block of tokens and of weight rows."""
    for n, m, d in ((7, 72, 2176), (13, 4200, 384), (20, 72, 640), (50, 88, 2176), (70, 2200, 640), (200, 2200, 2176), (1100, 520, 384)):
        c = Case(orbq, n, m, d, ba, bw, 2, [0, n // 3, n], seed=5)
        for name in ("f32", "bf16"):
            c.check(c.call(ALL, "gelu_tanh", name), ALL, "gelu_tanh", name)


def test_either_side_of_the_few_rows(orbq):
    """64 and 65 tokens, and sizes of which the tiles take some and the few-row form the others."""
    for n, m, d in ((64, 520, 256), (65, 520, 256), (64, 16400, 256), (65, 16400, 256), (300, 6000, 128), (800, 6000, 128), (4096, 64, 128),
                    (4097, 64, 128)):
        c = Case(orbq, n, m, d, 4, 4, 1, None, seed=6)
        c.check(c.call(ALL, "none", "bf16"), ALL, "none", "bf16")


# more rows than the few-row form has: tiles, of either shape, whole and ragged, with an odd count of K tiles
TILES = [(4100, 72, 320, 4, 4, 2, None), (4608, 192, 256, 4, 4, 1, None), (5000, 256, 192, 2, 4, 2, None), (4300, 520, 448, 3, 3, 3, [0, 100, 100, 4300]),
         (4400, 760, 256, 6, 4, 4, [7, 300, 1500, 2700, 4390]), (4200, 1000, 128, 4, 2, 4200, None), (4700, 264, 576, 6, 6, 2, None),
         (4097, 8, 64, 4, 6, 1, None), (6000, 1536, 192, 2, 2, 3, [0, 900, 1900, 6000])]


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,d,ba,bw,groups,cu", TILES)
def test_tiles(orbq, n, m, d, ba, bw, groups, cu, name):
    log(f"lut_gemm fused tiles {name} n={n} m={m} d={d} A{ba} W{bw} groups={groups} cu={cu}")
    c = Case(orbq, n, m, d, ba, bw, groups, cu, vectors="f32" if n % 2 else "bf16", seed=7)
    for parts, act in ((ALL, "none"), (("bias",), "gelu_tanh"), (("gate", "residual"), "gelu_erf")):
        c.check(c.call(parts, act, name), parts, act, name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_tiles_in_place(orbq, name):
    """Tiles that write a part of a wider tensor, onto the residual, and leave rows alone."""
    torch = torch_mod()
    n, m, d = 4300, 200, 192
    c = Case(orbq, n, m, d, 4, 4, 3, [2, n // 2, n // 2, n - 3], seed=8)
    want = c.call(ALL, "gelu_tanh", name)
    res = torch.full((n, m + 24), 7.0, dtype=dtype_of(name), device="cuda")
    r, rows = res[:, :m], slice(2, n - 3)
    r.copy_(c.t["residual"][name])
    before = r.clone()
    c.t["residual"][name] = r
    assert c.call(ALL, "gelu_tanh", name, out=r) is r
    assert torch.equal(r[rows], want[rows]) and torch.equal(r[:2], before[:2]) and torch.equal(r[n - 3:], before[n - 3:])
    assert bool((res[:, m:] == 7).all())
    c.cu = [9, -4, 2 ** 31 - 1, 1]
    c.call(ALL, "none", name, out=r)
    assert bool((res[:, m:] == 7).all())


@pytest.mark.parametrize("ba,bw", [(2, 2), (3, 3), (4, 4), (6, 6), (4, 6), (6, 2)])
def test_half_a_super_step(orbq, ba, bw):
    """Depths that are odd multiples of 64 in every few-row form."""
    for n, m, d in ((7, 72, 64), (13, 4200, 192), (20, 72, 2112), (50, 88, 704), (70, 2200, 320), (200, 2200, 448)):
        c = Case(orbq, n, m, d, ba, bw, 2, [0, n // 3, n], seed=9)
        for name in ("f32", "bf16"):
            c.check(c.call(ALL, "gelu_tanh", name), ALL, "gelu_tanh", name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,d", [(9, 104, 256), (64, 1000, 128), (200, 104, 256), (800, 1000, 128)])
def test_strides_in_place_and_rows_left_alone(orbq, n, m, d, name):
    torch = torch_mod()
    c = Case(orbq, n, m, d, 4, 4, 3, [2, n // 2, n // 2, n - 3])
    want = c.call(ALL, "gelu_tanh", name)
    wide, res = (torch.full((n, m + 24), 7.0, dtype=dtype_of(name), device="cuda") for _ in range(2))
    y, r = wide[:, :m], res[:, :m]
    r.copy_(c.t["residual"][name])
    c.t["residual"][name] = r
    assert c.call(ALL, "gelu_tanh", name, out=y) is y
    c.check(y, ALL, "gelu_tanh", name)
    rows = slice(2, n - 3)
    assert torch.equal(y[rows], want[rows]) and bool((wide[:, m:] == 7).all()) and bool((wide[:2] == 7).all()) and bool((wide[n - 3:] == 7).all())
    before = r.clone()
    c.call(ALL, "gelu_tanh", name, out=r)            # Y += ...
    assert torch.equal(r[rows], want[rows]) and torch.equal(r[:2], before[:2]) and torch.equal(r[n - 3:], before[n - 3:])
    assert bool((res[:, m:] == 7).all())
    # whatever the bounds hold, nothing outside is touched
    c.cu = [9, -4, 2 ** 31 - 1, 1]
    c.call(ALL, "none", name, out=y)
    assert bool((wide[:, m:] == 7).all())


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf"])
def test_nothing_more_gives_the_products_bits(orbq, act):
    torch = torch_mod()
    for n, m, d, ba, bw in ((65, 200, 256, 4, 4), (500, 1000, 192, 3, 3), (1000, 264, 320, 6, 4), (16, 72, 64, 2, 6)):
        c = Case(orbq, n, m, d, ba, bw, 1, [0, n])
        for name in ("f32", "bf16"):
            plain = orbq.lut_gemm(*c.x, c.cb_a, *c.w, c.cb_w, d, out_dtype=dtype_of(name), act=act)
            assert torch.equal(c.call((), act, name), plain)


@pytest.mark.parametrize("n,m,d,ba,bw", [(5, 200, 256, 4, 4), (300, 200, 256, 4, 4), (40, 2048, 256, 6, 4), (100, 2056, 320, 6, 4), (100, 2000, 256, 6, 6)])
def test_linear(orbq, n, m, d, ba, bw):
    """The layer is its quantizer and the fused product, bit for bit (6-bit activations kept as centroids included)."""
    torch = torch_mod()
    c = Case(orbq, n, m, d, ba, bw, 1, None, seed=2)
    perm, signs = workloads.rotation(d)
    rot = orbq.Rotation.create(d, 64, perm, signs)
    x = torch.randn((n, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    c.x = orbq.rpbh_quantize(x, rot, c.cb_a)
    for name in ("bf16", "f32"):
        got = orbq.linear(x, rot, c.cb_a, *c.w, c.cb_w, out_dtype=dtype_of(name), act="gelu_tanh", **c.how(ALL, name))
        assert torch.equal(got, c.call(ALL, "gelu_tanh", name))


@pytest.mark.parametrize("n,m,d,bw,block,passes", [(2, 200, 256, 4, 128, 1), (16, 88, 512, 2, 64, 1), (37, 1001, 384, 3, 64, 1), (5, 130, 256, 6, 128, 2),
                                                   (1, 7, 128, 4, 128, 1)])
def test_linear_a16(orbq, n, m, d, bw, block, passes):
    torch = torch_mod()
    groups = n if n < 10 else 1
    c = Case(orbq, n, m, d, 4, bw, groups, None, seed=3, x=False)
    perm, signs = workloads.rotation_passes(d, passes)
    rot = orbq.Rotation.create(d, block, perm, signs, passes=passes)
    x = torch.randn((n, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    pi = dense_pi(d, block) if passes == 1 else oracle.rpbh_composed(d, block, perm, signs, passes)
    xr = x.double().cpu().numpy() @ pi.T
    size = np.abs(xr) @ np.abs(c.b).T
    args = (x, rot, *c.w, c.cb_w)
    for name in ("bf16", "f32"):
        for parts, act in ((ALL, "none"), (("bias",), "gelu_erf"), (("gate", "residual"), "gelu_tanh")):
            got = orbq.linear_a16(*args, out_dtype=dtype_of(name), act=act, **c.how(parts, name))
            # the rotated tokens are rounded to bf16 (2^-8 at most), as orbq_linear_a16's
            c.check(got, parts, act, name, xr @ c.b.T, size, rel=2.0 ** -8 + (d / 8 + 40) * E)
        plain = orbq.linear_a16(*args, out_dtype=dtype_of(name))
        whole = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        assert torch.equal(orbq.linear_a16(*args, out_dtype=dtype_of(name), cu=whole), plain)
    y = c.t["residual"]["f32"].clone()
    orbq.linear_a16(*args, out=y, residual=y, bias=c.t["bias"])
    assert torch.equal(y, orbq.linear_a16(*args, residual=c.t["residual"]["f32"], bias=c.t["bias"]))


def test_graph_of_tiles(orbq):
    torch = torch_mod()
    c = Case(orbq, 4200, 72, 192, 4, 4, 2, [0, 1400, 4200], seed=10)
    how, y = c.how(ALL, "bf16"), torch.empty((4200, 72), dtype=torch.bfloat16, device="cuda")
    call = lambda out: orbq.lut_gemm(*c.x, c.cb_a, *c.w, c.cb_w, 192, out=out, act="gelu_erf", **how)  # noqa: E731
    call(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y)
    for k in range(3):
        how["residual"].add_(1)
        how["cu"].copy_(torch.tensor([0, 1400 + k, 4200], dtype=torch.int32))
        graph.replay()
        assert torch.equal(y, call(torch.empty_like(y)))


def test_no_rows_and_no_columns(orbq):
    torch = torch_mod()
    c = Case(orbq, 8, 16, 128, 4, 4, 2)
    e = torch.empty
    got = orbq.lut_gemm(c.x[0][:0], c.x[1][:0], c.cb_a, *c.w, c.cb_w, 128, bias=c.t["bias"], residual=e((0, 16), device="cuda"))
    assert got.shape == (0, 16)
    got = orbq.lut_gemm(*c.x, c.cb_a, c.w[0][:0], c.w[1][:0], c.cb_w, 128, bias=e((0,), device="cuda"), gate=e((2, 0), device="cuda"))
    assert got.shape == (8, 0)


def test_graph(orbq):
    """Captured calls follow what their operands and the groups' bounds hold."""
    torch = torch_mod()
    cases = [Case(orbq, n, 200, 256, 4, 4, 2, [0, n // 3, n]) for n in (9, 300)]
    how = [c.how(ALL, "bf16") for c in cases]
    call = lambda c, h, y: orbq.lut_gemm(*c.x, c.cb_a, *c.w, c.cb_w, 256, out=y, act="gelu_tanh", **h)  # noqa: E731
    ys = [torch.empty((c.n, 200), dtype=torch.bfloat16, device="cuda") for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, h, y in zip(cases, how, ys):
            call(c, h, y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, h, y in zip(cases, how, ys):
            call(c, h, y)
    for k in range(3):
        for c, h in zip(cases, how):
            h["residual"].add_(1)
            h["cu"].copy_(torch.tensor([0, c.n // 3 + k, c.n], dtype=torch.int32))
        graph.replay()
        for c, h, y in zip(cases, how, ys):
            assert torch.equal(y, call(c, h, torch.empty_like(y)))


def test_more_codes_than_a_launch_addresses(orbq):
    """Beyond 2^31 bytes of activation codes the rows go out in several launches, each with its own part of the gate's groups and
    of the residual."""
    torch = torch_mod()
    d, m, block = 16384, 8, 1024
    n = (1 << 31) // (d // 2) + 2 * block
    c = Case(orbq, block, m, d, 4, 4, 1, None, seed=4)
    x = c.x[0].repeat(n // block, 1), c.x[1].repeat(n // block)
    gate = torch.arange(1, n // block + 1, device="cuda").float()[:, None].expand(-1, m).contiguous()
    res = torch.arange(n, device="cuda").float()[:, None].expand(-1, m).contiguous()
    plain = orbq.lut_gemm(*c.x, c.cb_a, *c.w, c.cb_w, d, cu=torch.tensor([0, block], dtype=torch.int32, device="cuda"))
    got = orbq.lut_gemm(*x, c.cb_a, *c.w, c.cb_w, d, gate=gate, residual=res)
    # gate times the product, rounded, plus the residual, rounded
    want = plain.repeat(n // block, 1) * gate.repeat_interleave(block, 0) + res
    assert torch.equal(got, want)


def test_refusals(orbq):
    torch = torch_mod()
    c = Case(orbq, 8, 64, 128, 4, 4, 2)
    t = {"bias": c.t["bias"], "gate": c.t["gate"], "residual": c.t["residual"]["f32"]}
    call = lambda **kw: orbq.lut_gemm(*c.x, c.cb_a, *c.w, c.cb_w, 128, **kw)  # noqa: E731
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [dict(bias=t["bias"][:32]), dict(bias=t["bias"].half()), dict(bias=t["bias"].cpu()), dict(gate=t["gate"][:, :32]),
           dict(gate=torch.ones(3, 64, device="cuda")), dict(gate=t["gate"].half()), dict(residual=t["residual"][:4]),
           dict(residual=t["residual"].bfloat16(), out_dtype=torch.float32), dict(residual=t["residual"][:, ::2], bias=t["bias"]),
           dict(cu=cu.long()), dict(cu=cu[:1]), dict(cu=cu.cpu()), dict(cu=torch.zeros(2, dtype=torch.int32, device="cuda"), gate=t["gate"]),
           dict(residual=torch.empty((8, 65), device="cuda")[:, 1:]), dict(residual=torch.empty((8, 66), device="cuda")[:, :64])]
    for kw in bad:
        with pytest.raises(orbq.OrbqError):
            call(**kw)
    with pytest.raises(ValueError):
        call(bias=t["bias"], act="relu")
    for a in ("bias", "gate", "residual"):
        leaf = t[a].clone().requires_grad_()
        y = call(**{a: leaf})
        assert torch.equal(y, call(**{a: t[a]}))
        with pytest.raises(orbq.OrbqError):
            y.sum().backward()
        with torch.no_grad():
            assert not call(**{a: leaf}).requires_grad
