"""The norms around a block on the GPU against the float64 oracle (oracle/block_norm.py).

Tolerances, from the arithmetic before any run; e = 2^-24, all relative to the values that the kernel reads:
  * a sum over a row is taken in at most 32 + 4 + 3 + 16 steps, so it is off by 64 e of the sum of magnitudes;
  * a normalised entry is off by f e (|v| + |mean| + 64 mean |v|) from its difference, and 64 e relative from the factor (half the
    error of the sum of squares, root and quotient, what the mean's error does to the variance): `off`;
  * r: |gate post_weight| off(y), and 4 e of each term; then half a step of the stream's type;
  * h, from the r that the kernel stored: |weight (1 + scale)| off(r), and 4 e of each term; half a step of the branch's type;
  * gradients: the same carried through the formulas (`through` below); sums over rows take at most their number of steps.
A step is 2^-8 (bf16), 2^-11 (f16) or 2^-24 (f32) of the value at most, half of eps.
"""
import numpy as np
import pytest

from oracle import block_norm as ob
from tests.gpu_common import log, torch_mod

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
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


def dev(x, name):
    """numpy -> GPU tensor of the type, and the float64 values it holds."""
    t = torch_mod().from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype_of(name)).cuda()
    return t, host(t)


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def off(v, kind, eps):
    """Bound of a normalised row's error."""
    if kind is None:
        return np.zeros_like(v)
    m = v.mean(-1, keepdims=True) if kind == "layer" else 0.0 * v[..., :1]
    f = 1.0 / np.sqrt(((v - m) ** 2).mean(-1, keepdims=True) + eps)
    raw = f * E * (np.abs(v) + np.abs(m) + 64 * np.abs(v).mean(-1, keepdims=True)) if kind == "layer" else 0.0
    return raw + 72 * E * np.abs((v - m) * f)


def per_row(v, groups, n, cu, default):
    """A vector [d], [1, d] or [groups, d] as rows [n, d]."""
    d = 1 if v is None else v.shape[-1]
    out = np.full((n, d), default)
    if v is not None:
        for g, rows in enumerate(ob.groups_of(n, groups, cu)):
            out[list(rows)] = ob.row_of(v, g, default)
    return out


def close(got, want, tol, name, what):
    got = host(got)
    tol = tol + UNIT[name] * np.abs(want) * (1 + 1e-6) + LEAST[name]
    err = np.abs(got - want)
    ok = err <= tol
    if not ok.all():
        at = np.unravel_index(np.argmax(np.where(ok, 0, err / tol)), err.shape)
        raise AssertionError(f"{what}: {got[at]} for {want[at]} at {at}, {(err / tol)[at]:.3g} of the tolerance; {np.sum(~ok)} of {ok.size}")


class Case:
    """Inputs of a call, on the GPU (t) and as float64 (v)."""

    def __init__(self, n, d, groups, cu, stream, branch, mod, norm, post, residual=True, weights=True, gate=True, shared=False, seed=0):
        rng = np.random.default_rng([seed, n, d])
        self.n, self.d, self.groups, self.cu, self.norm, self.post = n, d, groups, cu, norm, post if residual else None
        self.stream, self.branch, self.mod, self.eps = stream, branch, mod, 1e-5
        rows = lambda scale, mean=0.0: rng.standard_normal((n, d)) * scale * np.exp(0.5 * rng.standard_normal(d)) + mean  # noqa: E731
        raw = {"x": (rows(2.0, 0.7), stream), "y": (rows(1.0, -0.3), branch) if residual else None,
               "dr": (rows(1.0), stream), "dh": (rows(1.0, 0.2), branch)}
        m = rng.standard_normal((1 if shared else groups, 5, d)) * 0.5
        self.t, self.v = {}, {}
        for a, x in raw.items():
            self.t[a], self.v[a] = dev(*x) if x else (None, None)
        mods, mods64 = dev(m, mod)               # slices of one tensor
        for i, a in ((1, "gate"), (2, "scale"), (4, "shift")):
            there = (gate and residual) if a == "gate" else norm is not None
            self.t[a], self.v[a] = (mods[:, i], mods64[:, i]) if there else (None, None)
        for a, there in (("weight", weights and norm is not None), ("post_weight", weights and self.post is not None)):
            self.t[a], self.v[a] = dev(1 + 0.3 * rng.standard_normal(d), branch) if there else (None, None)

    def how(self, t=None):
        t = t or self.t
        cu = None if self.cu is None else torch_mod().tensor(self.cu, dtype=torch_mod().int32, device="cuda")
        return dict({a: t[a] for a in ("y", "gate", "weight", "scale", "shift", "post_weight")}, norm=self.norm, post=self.post,
                    eps=self.eps, cu=cu)

    def inside(self):
        return [i for g in ob.groups_of(self.n, self.groups, self.cu) for i in g]

    def check_forward(self, r, h):
        v, at = self.v, self.inside()
        ld = lambda a, default: per_row(v[a], self.groups, self.n, self.cu, default)[at]  # noqa: E731
        if v["y"] is not None:
            want = ob.stream(v["x"], v["y"], v["gate"], v["post_weight"], self.post, self.eps, self.groups, self.cu)[at]
            c = np.abs(ld("gate", 1.0) * (1.0 if v["post_weight"] is None else v["post_weight"]))
            z = np.stack([ob.unit(row, self.post, self.eps)[0] for row in v["y"][at]])
            close(r[at], want, c * (off(v["y"][at], self.post, self.eps) + 4 * E * np.abs(z)) + 4 * E * np.abs(v["x"][at]), self.stream, "r")
        if self.norm is None:
            assert h is None
            return
        r64 = host(r)
        want = ob.normed(r64, v["weight"], v["scale"], v["shift"], self.norm, self.eps, self.groups, self.cu)[at]
        c = np.abs((1.0 if v["weight"] is None else v["weight"]) * (1 + np.abs(ld("scale", 0.0))))
        z = np.stack([ob.unit(row, self.norm, self.eps)[0] for row in r64[at]])
        close(h[at], want, c * (off(r64[at], self.norm, self.eps) + 4 * E * np.abs(z)) + 4 * E * np.abs(ld("shift", 0.0)), self.branch, "h")

    def check_backward(self, r64, got, with_dr=True):
        v, n, at = self.v, self.n, self.inside()
        normed = self.norm is not None
        want = ob.gradients(r64, v["dr"] if with_dr else None, v["dh"] if normed else None, v["y"], v["gate"], v["weight"], v["scale"],
                            v["post_weight"], self.norm, self.post, self.eps, self.eps, self.groups, self.cu)
        rows = lambda a, default: per_row(v[a], self.groups, n, self.cu, default)  # noqa: E731
        mean = lambda x: np.abs(x).mean(-1, keepdims=True)  # noqa: E731

        def through(x, t, dt, kind):
            """(|gradient through the norm|'s parts, its error) from t and its error dt"""
            if kind is None:
                return dt
            z, f = (np.stack(a) for a in zip(*[ob.unit(row, kind, self.eps) for row in x]))
            f, dz = f[:, None], off(x, kind, self.eps)
            m = mean(t * z)
            err = dt + mean(dt) + 64 * E * mean(t) + dz * m + np.abs(z) * ((np.abs(t) * dz + dt * np.abs(z)).mean(-1, keepdims=True) + 64 * E * m)
            return f * (err + 80 * E * (np.abs(t) + mean(t) + np.abs(z) * m))

        dx = 4 * E * np.abs(v["dr"]) if with_dr else np.zeros((n, self.d))
        steps = n + 64
        group_sum = lambda x: np.stack([x[list(g)].sum(0) for g in ob.groups_of(n, self.groups, self.cu)])  # noqa: E731
        one = lambda x: 1.0 if x is None else np.abs(x)  # noqa: E731
        outside = [i for i in range(n) if i not in set(at)]
        if normed:
            s = 1 + np.abs(rows("scale", 0.0))
            t = np.abs(v["dh"] * one(v["weight"]) * s)
            dx = dx + through(r64, t, 4 * E * t, self.norm)
            z = np.stack([ob.unit(row, self.norm, self.eps)[0] for row in r64])
            size, err = np.abs(v["dh"] * z), np.abs(v["dh"]) * off(r64, self.norm, self.eps)
            self.check_vector("scale", got.scale, want["scale"], group_sum(err + steps * E * size) * one(v["weight"]) + 4 * E * np.abs(want["scale"]))
            self.check_vector("shift", got.shift, want["shift"], group_sum(steps * E * np.abs(v["dh"])))
            if v["weight"] is not None:
                close(got.weight, want["weight"], ((err + (steps + 8) * E * size) * s)[at].sum(0), self.branch, "dweight")
        dx[outside] = 0
        close(got.x, want["x"], dx, self.stream, "dx")
        if v["y"] is None:
            return
        c, pw = np.abs(rows("gate", 1.0)), one(v["post_weight"])
        q, z = np.abs(want["x"]), np.stack([ob.unit(row, self.post, self.eps)[0] for row in v["y"]])
        dy = through(v["y"], q * c * pw, (dx + 4 * E * q) * c * pw, self.post)
        dy[outside] = 0
        close(got.y, want["y"], dy, self.branch, "dy")
        size, err = np.abs(q * z), dx * np.abs(z) + q * off(v["y"], self.post, self.eps)
        self.check_vector("gate", got.gate, want["gate"], group_sum(err + steps * E * size) * pw + 4 * E * np.abs(want["gate"]))
        if v["post_weight"] is not None:
            close(got.post_weight, want["post_weight"], ((err + (steps + 8) * E * size) * c)[at].sum(0), self.branch, "dpost_weight")

    def check_vector(self, name, got, want, tol):
        if self.v[name] is None:
            assert got is None
            return
        if self.v[name].shape[0] == 1 and self.groups > 1:      # shared by the groups
            want, tol = want.sum(0, keepdims=True), tol.sum(0, keepdims=True) + self.groups * E * np.abs(want).sum(0, keepdims=True)
        close(got, want, tol, self.mod, "d" + name)


TYPES = [("bf16", "bf16", "f32"), ("f16", "f16", "f16"), ("f32", "bf16", "f32"), ("f32", "f32", "f32"), ("f32", "f16", "f16"),
         ("bf16", "bf16", "bf16")]
CASES = [
    # n, d, groups, cu, types, norm, post
    (1, 1536, 1, None, 0, "layer", None), (48, 1536, 48, None, 5, "layer", None), (37, 1536, 1, None, 2, "rms", "rms"),
    (21, 1, 3, None, 0, "rms", "rms"), (5, 7, 1, None, 3, "layer", "layer"), (12, 8, 4, None, 4, "layer", "rms"),
    (130, 128, 2, None, 1, "rms", None), (70, 100, 5, [2, 2, 30, 31, 60, 64], 0, "layer", "layer"), (33, 512, 1, None, 3, "layer", "rms"),
    (33, 520, 3, None, 2, "rms", "layer"), (9, 1000, 1, None, 5, "layer", None), (10, 1024, 2, [0, 7, 10], 1, "layer", "rms"),
    (11, 1537, 1, None, 2, "layer", "rms"), (6, 2048, 3, [0, 1, 1, 6], 4, "rms", "rms"), (7, 2056, 1, None, 0, "layer", "layer"),
    (19, 4096, 2, [3, 4, 19], 5, "rms", "rms"), (5, 4100, 1, None, 3, "layer", None), (4, 5000, 2, None, 1, "layer", "layer"),
    (3, 8192, 1, None, 2, "rms", "layer"), (6, 8200, 3, None, 0, "layer", "rms"), (3, 12289, 1, None, 5, "layer", "rms"),
    (4, 16384, 2, None, 4, "layer", "layer"), (2, 16384, 1, None, 5, "rms", None), (3001, 64, 7, [0, 0, 1, 2, 900, 901, 3000, 3000], 0, "layer", "rms"),
    (2500, 24, 2500, None, 3, "rms", None), (40, 320, 1, None, 0, None, "rms"), (40, 33, 8, None, 2, None, None)]


@pytest.mark.parametrize("n,d,groups,cu,types,norm,post", CASES)
def test_both_ways(orbq, n, d, groups, cu, types, norm, post):
    log(f"block_norm n={n} d={d} groups={groups} cu={cu} {TYPES[types]} {norm} {post}")
    c = Case(n, d, groups, cu, *TYPES[types], norm, post)
    r, h = orbq.block_norm(c.t["x"], dtype=dtype_of(c.branch), **c.how())
    c.check_forward(r, h)
    g = orbq.block_norm_backward(r, c.t["dh"] if norm else None, c.t["dr"], **c.how())
    if c.cu is not None:      # rows that no group has hold anything: the oracle does not look at them
        r = r.clone()
        r[[i for i in range(n) if i not in set(c.inside())]] = 0
    c.check_backward(host(r), g)


@pytest.mark.parametrize("types", range(len(TYPES)))
@pytest.mark.parametrize("d", [512, 1000, 1536, 2040, 4096, 8184, 16384, 509, 4001, 9001])
def test_every_form(orbq, d, types):
    """Each split of a row over registers, lanes and waves, in each type, with as many rows as make a workgroup take several."""
    log(f"block_norm forms d={d} {TYPES[types]}")
    for n, groups, cu, norm, post in ((1100, 2, [0, 500, 1100], "layer", "rms") if d < 1000 else (11, 2, [1, 4, 11], "layer", "rms"),
                                      (9, 3, None, "rms", "layer"), (5, 1, None, "layer", None), (6, 2, None, "rms", "rms"), (3, 1, None, "rms", None)):
        c = Case(n, d, groups, cu, *TYPES[types], norm, post, seed=types)
        r, h = orbq.block_norm(c.t["x"], dtype=dtype_of(c.branch), **c.how())
        c.check_forward(r, h)
        g = orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **c.how())
        if cu is not None and cu[0]:
            r = r.clone()
            r[:cu[0]] = 0
        c.check_backward(host(r), g)


@pytest.mark.parametrize("kw", [dict(residual=False), dict(residual=False, weights=False), dict(gate=False), dict(shared=True),
                                dict(gate=False, weights=False, shared=True)])
@pytest.mark.parametrize("norm,post", [("layer", "rms"), ("rms", None)])
def test_parts_that_are_missing_or_shared(orbq, kw, norm, post):
    for types, d in ((0, 256), (2, 150)):
        c = Case(60, d, 4, None, *TYPES[types], norm, post, **kw)
        r, h = orbq.block_norm(c.t["x"], dtype=dtype_of(c.branch), **c.how())
        if c.t["y"] is None:
            assert r is c.t["x"]
        c.check_forward(r, h)
        c.check_backward(host(r), orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **c.how()))
        c.check_backward(host(r), orbq.block_norm_backward(r, c.t["dh"], None, **c.how()), with_dr=False)


@pytest.mark.parametrize("d", [1536, 300, 4096])
def test_rows_do_not_depend_on_the_call(orbq, d):
    """A row alone, among others, strided, in place and with a shared vector: the same bits."""
    torch = torch_mod()
    c = Case(50, d, 1, None, "bf16", "bf16", "bf16", "layer", "rms")
    how = c.how()
    r, h = orbq.block_norm(c.t["x"], **how)
    for i in (0, 17, 49):
        one = orbq.block_norm(c.t["x"][i:i + 1], **dict(how, y=c.t["y"][i:i + 1]))
        assert torch.equal(one[0][0], r[i]) and torch.equal(one[1][0], h[i])
    for pad in (8, 1):       # 16-byte columns, and not
        wide = [torch.full((50, d + pad), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        x, y, rr, hh = (w[:, :d] for w in wide)
        x.copy_(c.t["x"])
        y.copy_(c.t["y"])
        got = orbq.block_norm(x, out=(rr, hh), **dict(how, y=y))
        assert got[0] is rr and got[1] is hh
        if pad == 8:
            assert torch.equal(rr, r) and torch.equal(hh, h)
        else:                # another split of a row's sums
            c.check_forward(rr, hh)
        assert all(bool((w[:, d:] == 7.0).all()) for w in wide)
        got = orbq.block_norm(x, out=(x, y), **dict(how, y=y))        # in place
        assert got[0] is x and torch.equal(x, rr) and torch.equal(y, hh)
    # the norm of the stored stream, by a call of its own, is the same norm
    alone = orbq.block_norm(r, weight=how["weight"], scale=how["scale"], shift=how["shift"], norm="layer", eps=c.eps)
    assert torch.equal(alone[1], h)
    # gradients in place
    g = orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **how)
    for _ in range(2):       # the sums do not depend on scheduling
        again = orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **how)
        assert all(torch.equal(a, b) for a, b in zip(g, again))


def test_rows_outside_the_groups_are_left_alone(orbq):
    torch = torch_mod()
    c = Case(40, 128, 3, [5, 9, 9, 30], "bf16", "bf16", "f32", "rms", "rms")
    r, h = (torch.full((40, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = c.t["x"].clone()
    x[:5] = float("nan")
    y = c.t["y"].clone()
    y[30:] = float("inf")
    orbq.block_norm(x, out=(r, h), **dict(c.how(), y=y))
    c.check_forward(r, h)
    for t in (r, h):
        assert bool((t[:5] == 3).all()) and bool((t[30:] == 3).all())
    g = orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **c.how())
    assert not g.x[:5].any() and not g.x[30:].any() and not g.y[:5].any() and not g.y[30:].any()
    assert not g.gate[1].any() and not g.scale[1].any() and g.gate[0].any()
    # whatever the bounds hold, nothing outside the buffers is touched and every row is done once at most
    bad = dict(c.how(), cu=torch.tensor([7, -3, 2 ** 31 - 1, 12], dtype=torch.int32, device="cuda"))
    orbq.block_norm(c.t["x"], **bad)
    orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **bad)
    torch.cuda.synchronize()


def test_special_values(orbq):
    """Zero rows, infinities and NaN stay in their rows; an infinite sum of squares gives zeros or NaN, not garbage elsewhere."""
    torch = torch_mod()
    c = Case(8, 256, 1, None, "f32", "f32", "f32", "layer", "rms")
    x, y = c.t["x"].clone(), c.t["y"].clone()
    x[1], y[1] = 0, 0
    x[2, 3], y[3, 5], x[4, 0] = float("nan"), float("inf"), -float("inf")
    r, h = orbq.block_norm(x, **dict(c.how(), y=y))
    assert torch.isfinite(h[[0, 1, 5, 6, 7]]).all()
    assert torch.equal(r[1], torch.zeros_like(r[1])) and torch.equal(h[1], c.t["shift"][0])
    assert torch.isnan(h[2:5]).all()
    want = orbq.block_norm(c.t["x"], **c.how())
    assert all(torch.equal(a[[0, 5, 6, 7]], b[[0, 5, 6, 7]]) for a, b in zip((r, h), want))


def test_no_rows(orbq):
    torch = torch_mod()
    x = torch.empty((0, 64), device="cuda")
    v = torch.ones((3, 64), device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    r, h = orbq.block_norm(x, x, gate=v, scale=v, shift=v, cu=cu)
    assert r.shape == h.shape == (0, 64)
    g = orbq.block_norm_backward(x, x, x, y=x, gate=v, scale=v, shift=v, cu=cu)
    assert g.x.shape == (0, 64) and not g.gate.any() and g.gate.shape == (3, 64)
    leaf = v.clone().requires_grad_()
    orbq.block_norm(x, x, gate=leaf, cu=cu)[1].sum().backward()
    assert not leaf.grad.any()


@pytest.mark.parametrize("shape", ["groups", "shared", "expanded"])
@pytest.mark.parametrize("norm,post", [("layer", "rms"), ("rms", None), (None, "layer")])
def test_autograd(orbq, shape, norm, post):
    """Leaves get what the backward entry point gives, also where one output is unused and a vector is broadcast."""
    torch = torch_mod()
    c = Case(24, 96, 3, None, "f32", "f32", "f32", norm, post, shared=shape == "shared")
    names = [a for a in ("x", "y", "gate", "weight", "scale", "shift", "post_weight") if c.t[a] is not None]
    leaf = {a: c.t[a].clone().requires_grad_() for a in names}
    if shape == "expanded":
        for a in ("gate", "scale", "shift"):
            if a in leaf:
                leaf[a] = c.t[a][0].clone().requires_grad_()
    t = dict(c.t, **leaf)
    if shape == "expanded":
        t.update({a: t[a][None].expand(3, 96) for a in ("gate", "scale", "shift") if a in leaf})
    r, h = orbq.block_norm(t["x"], **c.how(t))
    loss = (r * c.t["dr"]).sum() + ((h * c.t["dh"]).sum() if norm else 0)
    loss.backward()
    plain = {a: (None if x is None else x.detach()) for a, x in t.items()}
    g = orbq.block_norm_backward(r.detach(), c.t["dh"] if norm else None, c.t["dr"], **c.how(plain))
    for a in names:
        want = getattr(g, a)
        if shape == "expanded" and a in ("gate", "scale", "shift"):
            want = want.sum(0)
        assert torch.equal(leaf[a].grad, want), a
    # only some are asked for, and only one output is used (its gradient an expanded one)
    some = c.t["y"].clone().requires_grad_()
    r, h = orbq.block_norm(c.t["x"], **dict(c.how(), y=some))
    (r.sum() if norm is None else h.sum()).backward()
    ones = torch.ones_like(c.t["x"])
    g = orbq.block_norm_backward(r.detach(), ones if norm else None, None if norm else ones, **c.how())
    assert torch.equal(some.grad, g.y)
    if norm:
        r, h = orbq.block_norm(c.t["x"], **dict(c.how(), y=some))
        some.grad = None
        r.sum().backward()
        g = orbq.block_norm_backward(r.detach(), None, ones, **dict(c.how(), norm=None, weight=None, scale=None, shift=None))
        assert torch.equal(some.grad, g.y)


def test_gradient_by_differences(orbq):
    """Against differences of the kernel's own forward pass, in 32 bits: a step of 2^-6 leaves an error of its square's
    order, 2^-12 of third derivatives, and 2^-23 2^6 of the loss's terms from rounding."""
    torch = torch_mod()
    c = Case(6, 40, 2, None, "f32", "f32", "f32", "layer", "rms")
    loss = lambda t: sum(float((a.double() * b.double()).sum()) for a, b in zip(orbq.block_norm(t["x"], **c.how(t)), (c.t["dr"], c.t["dh"])))  # noqa: E731
    r, _ = orbq.block_norm(c.t["x"], **c.how())
    g = orbq.block_norm_backward(r, c.t["dh"], c.t["dr"], **c.how())
    rng = np.random.default_rng(3)
    for a in ("x", "y", "gate", "weight", "scale", "shift", "post_weight"):
        way = torch.from_numpy(rng.standard_normal(tuple(c.t[a].shape))).float().cuda()
        way /= way.norm()
        up, down = (dict(c.t, **{a: (c.t[a] + s * 2.0 ** -6 * way)}) for s in (1, -1))
        want = (loss(up) - loss(down)) / 2.0 ** -5
        got = float((getattr(g, a).double() * way.double()).sum())
        assert abs(got - want) < 0.01 * (1 + abs(want)), (a, got, want)


def test_streams_graphs_and_workspaces(orbq):
    """Captured calls follow what their inputs hold, also the groups' bounds, and share no scratch with eager calls."""
    torch = torch_mod()
    c = Case(700, 256, 3, [0, 100, 400, 700], "bf16", "bf16", "f32", "layer", "rms")
    how = c.how()
    x, dh, dr, cu = c.t["x"].clone(), c.t["dh"].clone(), c.t["dr"].clone(), how["cu"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r, h = orbq.block_norm(x, **how)
        g = orbq.block_norm_backward(r, dh, dr, **how)
    torch.cuda.current_stream().wait_stream(side)
    c.check_forward(r, h)
    c.check_backward(host(r), g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, h = orbq.block_norm(x, **how)
        g = orbq.block_norm_backward(r, dh, dr, **how)
    for k in range(3):
        x.copy_(c.t["x"] * (k + 1))
        cu.copy_(torch.tensor([k, 100 + k, 300, 700 - 50 * k], dtype=torch.int32))
        graph.replay()
        want_r, want_h = orbq.block_norm(x, **how)      # eager work between the replays
        want_g = orbq.block_norm_backward(want_r, dh, dr, **how)
        torch.cuda.synchronize()
        at = slice(k, 700 - 50 * k)
        assert torch.equal(r[at], want_r[at]) and torch.equal(h[at], want_h[at])
        assert all(torch.equal(a, b) for a, b in zip(g, want_g))


def test_refusals(orbq):
    torch = torch_mod()
    x = torch.randn(8, 64, device="cuda")
    v = torch.randn(2, 64, device="cuda")
    bad = [dict(x=x[0]), dict(x=x.double()), dict(x=x.cpu()), dict(x=x.t().contiguous().t()), dict(y=x[:4]), dict(y=x.bfloat16(), dtype=torch.float32),
           dict(norm="batch"), dict(post="batch"), dict(gate=v), dict(gate=v[:, :32]), dict(y=x, gate=v, scale=v.bfloat16()),
           dict(scale=torch.randn(3, 64, device="cuda")), dict(weight=v), dict(weight=v[0].cpu()), dict(post_weight=v[0]),
           dict(norm=None), dict(norm=None, y=x, shift=v), dict(eps=-1.0), dict(cu=torch.zeros(3, device="cuda")),
           dict(cu=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(out=(x, x[:, :32])), dict(out=(x, None)),
           dict(y=x, out=(x.bfloat16(), x)), dict(x=x.half(), dtype=torch.bfloat16), dict(dtype=torch.float64),
           dict(y=x, post="rms", weight=v[0], post_weight=v[0].half())]
    for kw in bad:
        with pytest.raises(orbq.OrbqError):
            orbq.block_norm(**{**dict(x=x), **kw})
    for args, kw in (((x, None), {}), ((x, x[:4]), {}), ((x, x.bfloat16()), dict(y=x)), ((x, x, x.half()), {}),
                     ((x, x), dict(norm=None)), ((x, None, x), {}), ((x, x), dict(workspace=torch.empty(64, device="cuda"), shift=v))):
        with pytest.raises(orbq.OrbqError):
            orbq.block_norm_backward(*args, **kw)
    leaf = x.clone().requires_grad_()
    g, = torch.autograd.grad(orbq.block_norm(leaf)[1].square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
