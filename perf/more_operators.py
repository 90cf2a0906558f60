"""Cases of a transformer block's operators around its quantized projections and its 8-bit cache: the norms
before and after a block with its gate and residual (and their gradients), the append to the cache that turns
q and k by their positions on the way, and the quantized products with bias, activation, gate and residual in
their epilogue.

`own = False` computes them in their plain form (elementary torch operations in 32 bits, angles in 64, rounded
once at the end); `own = True` calls the framework.  Sizes: the video layers' 21 x 30 x 52 latent tokens (1560 a
frame), width 1536 (12 heads of 128) and 8960 hidden; batched, image and token-by-token sizes are generic.
"""
from __future__ import annotations

import functools
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
SCALE_FLOOR = 2.0 ** -64      # the least scale of a block of the cache
GROW = 1.25                   # a block's scale that has to grow grows at least by this factor
INV127 = float(np.float32(1.0) / np.float32(127.0))


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # between two branches of a layer, one token each of 48 sequences with modulations of their own: latency
        {"name": "norm_step", "op": "norm", "n": 48, "d": 1536, "groups": 48, "ragged": False, "norm": "layer", "post": "",
         "residual": True, "weights": False, "stream": "bf16", "branch": "bf16", "mod": "bf16", "grad": False},
        # the same for a whole video clip, one modulation for all its tokens, which is kept in 32 bits
        {"name": "norm_video", "op": "norm", "n": 32760, "d": 1536, "groups": 1, "ragged": False, "norm": "layer", "post": "",
         "residual": True, "weights": False, "stream": "bf16", "branch": "bf16", "mod": "f32", "grad": False},
        # its gradient in training, the residual stream in 32 bits
        {"name": "norm_video_grad", "op": "norm", "n": 32760, "d": 1536, "groups": 1, "ragged": False, "norm": "layer",
         "post": "", "residual": True, "weights": False, "stream": "f32", "branch": "bf16", "mod": "f32", "grad": True},
        # gradient of a layer with a norm on either side of each branch, a ragged batch of images and their texts
        {"name": "norm_sandwich_grad", "op": "norm", "n": 9001, "d": 4096, "groups": 7, "ragged": True, "norm": "rms",
         "post": "rms", "residual": True, "weights": True, "stream": "bf16", "branch": "bf16", "mod": "bf16", "grad": True},
        # one token appended to each of 48 running sequences, q and k normalised and turned: latency
        {"name": "append_step", "op": "append", "batch": 48, "new": 1, "ragged": False, "held": 8000, "qh": 32, "kh": 8,
         "d": 128, "page": 64, "dims": "128", "layout": "halves", "dtype": "bf16", "norm": True},
        # three frames of a video behind the 18 held ones (and some text tokens), turned by time, row and column
        {"name": "append_frames", "op": "append", "batch": 1, "new": 4680, "ragged": False, "held": 28117, "qh": 12, "kh": 12,
         "d": 128, "page": 64, "dims": "44,42,42", "layout": "pairs", "dtype": "bf16", "norm": False},
        # prompts of a ragged batch in short blocks, narrow heads of which a part is turned
        {"name": "append_prompts", "op": "append", "batch": 7, "new": 5000, "ragged": True, "held": 0, "qh": 16, "kh": 4,
         "d": 64, "page": 16, "dims": "32", "layout": "halves", "dtype": "f16", "norm": True},
        # the modulation vectors of two samples, from 16-bit activations and 4-bit weights, with their bias: latency
        {"name": "product_vectors", "op": "product", "form": "a16", "n": 2, "k": 1536, "m": 9216, "ba": 16, "bw": 4,
         "act": "none", "bias": True, "gate": False, "residual": False, "groups": 1, "ragged": False, "out": "bf16"},
        # up-projection of a few new tokens of a running batch, one each of 5 sequences: latency
        {"name": "product_step", "op": "product", "form": "codes", "n": 5, "k": 1536, "m": 8960, "ba": 4, "bw": 4,
         "act": "gelu_tanh", "bias": True, "gate": False, "residual": False, "groups": 1, "ragged": False, "out": "bf16"},
        # up-projection of a video clip, bias and GELU
        {"name": "product_video_up", "op": "product", "form": "codes", "n": 32760, "k": 1536, "m": 8960, "ba": 4, "bw": 4,
         "act": "gelu_tanh", "bias": True, "gate": False, "residual": False, "groups": 1, "ragged": False, "out": "bf16"},
        # down-projection of the same onto the residual stream in 32 bits, bias and gate
        {"name": "product_video_down", "op": "product", "form": "codes", "n": 32760, "k": 8960, "m": 1536, "ba": 4, "bw": 4,
         "act": "none", "bias": True, "gate": True, "residual": True, "groups": 1, "ragged": False, "out": "f32"},
        # attention's output projection onto the residual stream, three samples of unequal length, gates of their own
        {"name": "product_out_ragged", "op": "product", "form": "codes", "n": 9210, "k": 1536, "m": 1536, "ba": 4, "bw": 4,
         "act": "none", "bias": True, "gate": True, "residual": True, "groups": 3, "ragged": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "append", "product"])
    if op == "norm":
        d = _log(rng, 8, 8192)
        d = d if rng.random() < 0.3 else (d + 7) // 8 * 8       # widths are multiples of 8 mostly
        n = _log(rng, 1, min(40000, 4 * 10 ** 7 // d))
        groups = rng.choice([1, _log(rng, 1, min(n, 64))])
        ragged = groups > 1 and rng.random() < 0.5
        stream, branch = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f32"), ("f32", "f16")])
        return {"op": "norm", "n": n if ragged else max(1, n // groups) * groups, "d": d, "groups": groups, "ragged": ragged,
                "norm": rng.choice(["layer", "rms"]), "post": rng.choice(["", "", "rms", "layer"]),
                "residual": rng.random() < 0.8, "weights": rng.random() < 0.5, "stream": stream, "branch": branch,
                "mod": rng.choice(["f32", branch]), "grad": rng.random() < 0.5}
    if op == "append":
        kh, d, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
        dims = {64: ["64", "32", "16,24,24"], 128: ["128", "44,42,42", "64"], 256: ["256", "64,64,64", "64"]}[d]
        batch = _log(rng, 1, 64)
        return {"op": "append", "batch": batch, "new": _log(rng, 1, 4096 // batch), "ragged": rng.random() < 0.5,
                "held": rng.choice([0, _log(rng, 1, 4096)]), "qh": kh * rng.choice([1, 2, 4]), "kh": kh, "d": d, "page": page,
                "dims": rng.choice(dims), "layout": rng.choice(["pairs", "halves"]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "norm": rng.random() < 0.5}
    form = rng.choice(["codes", "codes", "codes", "a16"])
    k = 128 * _log(rng, 2, 70) if form == "a16" else 64 * _log(rng, 4, 140)
    m = 8 * _log(rng, 16, 1150)
    n = _log(rng, 1, 64) if form == "a16" else _log(rng, 1, min(20000, int(2e11 / (k * m))))
    ba, bw = rng.choice([(4, 4), (4, 2), (3, 3), (6, 4), (2, 2)])
    groups = rng.choice([1, _log(rng, 1, min(n, 16))])
    ragged = groups > 1 and rng.random() < 0.5
    return {"op": "product", "form": form, "n": n if ragged else max(1, n // groups) * groups, "k": k, "m": m,
            "ba": 16 if form == "a16" else ba, "bw": bw, "act": rng.choice(["none", "gelu_tanh", "gelu_erf"]),
            "bias": rng.random() < 0.8, "gate": rng.random() < 0.5, "residual": rng.random() < 0.5, "groups": groups,
            "ragged": ragged, "out": "bf16" if form == "a16" else rng.choice(["bf16", "bf16", "f32"])}


def _bounds(case):
    """First row of each group and the row behind the last: part of the case, not of the seed."""
    n, groups = case["n"], case["groups"]
    if not case["ragged"]:
        return [n // groups * i for i in range(groups)] + [n]
    rng = random.Random("%d %d" % (n, groups))
    return [0] + sorted(rng.randint(0, n) for _ in range(groups - 1)) + [n]     # some groups may have no rows


def _lengths(case):
    """(tokens before the call, new tokens) of each sequence: part of the case, not of the seed."""
    rng = random.Random("%(batch)d %(new)d %(d)d %(page)d" % case)
    n, h = case["new"], case["held"]
    new = [rng.randint(1, n) if case["ragged"] else n for _ in range(case["batch"])]
    return [rng.randint(h // 8, h) if case["batch"] > 1 else h for _ in range(case["batch"])], new


# ------------------------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "append": _prepare_append, "product": _prepare_product}[case["op"]](case, gen, seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_norm(case, gen, seed):
    n, d = case["n"], case["d"]
    stream, branch, mod = (DTYPES[case[a]] for a in ("stream", "branch", "mod"))
    # the residual stream has channels that stand out, and a mean
    x = _normal(gen, n, d).mul_(torch.exp(_normal(gen, d))).add_(0.5 * _normal(gen, d)).to(stream)
    s = {"case": case, "x": x, "y": _normal(gen, n, d).to(branch) if case["residual"] else None}
    # the modulations of a layer as its projection gives them: shift, scale, gate of two branches side by side
    v = (_normal(gen, case["groups"], 6, d) * 0.3).to(mod)
    s["gate"], s["shift"], s["scale"] = (v[:, 2] if case["residual"] else None), v[:, 3], v[:, 4]
    weights = (1 + 0.2 * _normal(gen, 2, d)).to(branch)
    s["weight"] = weights[0] if case["weights"] else None
    s["post_weight"] = weights[1] if case["weights"] and case["post"] and case["residual"] else None
    s["cu"] = _ints(_bounds(case)) if case["ragged"] else None
    if case["grad"]:       # x takes the part of the stream behind the branch, which the forward pass kept
        s["dr"], s["dh"] = _normal(gen, n, d).to(stream), _normal(gen, n, d).to(branch)
    return s


def _prepare_append(case, gen, seed):
    held, new = _lengths(case)
    batch, page, qh, kh, d, dt = case["batch"], case["page"], case["qh"], case["kh"], case["d"], DTYPES[case["dtype"]]
    lens = [a + b for a, b in zip(held, new)]
    per = [(x + page - 1) // page for x in lens]
    pages = sum(per) + 3                      # the last one is nobody's
    order = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed), dtype=torch.int64)
    table = torch.zeros((batch, max(per)), dtype=torch.int32)
    table[torch.arange(max(per)) < torch.tensor(per)[:, None]] = order[: sum(per)].int()
    total = sum(new)
    codes = lambda: torch.round(_normal(gen, pages, kh, page * d) * 30).clamp_(-127, 127).to(torch.int8)  # noqa: E731
    scales = lambda: torch.exp(0.3 * _normal(gen, pages, kh)) / 30  # noqa: E731
    dims = [int(x) for x in case["dims"].split(",")]
    where = np.concatenate([np.arange(h, h + n) for h, n in zip(held, new)])
    # one axis: the token's place in its sequence; three: time, row and column of 30 x 52 tokens a frame
    pos = where[:, None] if len(dims) == 1 else np.stack([where // 1560, where // 52 % 30, where % 52], 1)
    freqs = np.concatenate([10000.0 ** (-np.arange(0, k, 2) / k) for k in dims])
    first = [h // page * page for h in held]  # what is read back: the new tokens and the block they joined
    read = [x - f for x, f in zip(lens, first)]
    x = (_normal(gen, total, qh + 2 * kh, d) * torch.exp(0.3 * _normal(gen, total, qh + 2 * kh, 1))).to(dt)
    w = 1 + 0.2 * _normal(gen, 2, d)
    return {"case": case, "table": table.cuda(), "kc": codes().view(pages, kh, page, d), "vc": codes().view(pages, kh, d, page),
            "ks": scales(), "vs": scales(), "start": _ints(held), "cu": _ints([0] + np.cumsum(new).tolist()), "max_new": max(new),
            "dims": dims, "pos": torch.from_numpy(pos).float().cuda(), "freqs": torch.from_numpy(freqs).float().cuda(),
            # the parts of a fused projection, where they lie
            "q": x[:, :qh], "k": x[:, qh:qh + kh], "v": x[:, qh + kh:],
            "q_weight": w[0] if case["norm"] else None, "k_weight": w[1] if case["norm"] else None,
            "first": _ints(first), "cu_read": _ints([0] + np.cumsum(read).tolist()), "total_read": sum(read), "max_read": max(read)}


@functools.lru_cache(maxsize=None)
def _centroids(bits, d):
    """Centroids of a normal distribution of variance 1 / d, each the mean of its cell, in 32 bits and antisymmetric."""
    half = 1 << (bits - 1)
    t = np.linspace(0.0, 8.0, 160001)
    mass = np.exp(-t * t / 2)
    mass0, mass1 = np.concatenate([[0], np.cumsum(mass)]), np.concatenate([[0], np.cumsum(mass * t)])
    c = (np.arange(half) + 0.5) * (3.0 / half)
    for _ in range(400):
        at = np.concatenate([[0], np.searchsorted(t, (c[1:] + c[:-1]) / 2), [len(t)]])
        c = (mass1[at[1:]] - mass1[at[:-1]]) / (mass0[at[1:]] - mass0[at[:-1]])
    c = (c / math.sqrt(d)).astype(np.float32)
    return np.concatenate([-c[::-1], c])


def _pack(codes, bits):
    """Codes of `bits` bits [rows, d] as bytes, the first in the least significant bits: 8 codes are `bits` bytes."""
    rows, d = codes.shape
    word = (codes.view(rows, d // 8, 8).long() << (bits * torch.arange(8, device="cuda"))).sum(-1)
    return (word[..., None] >> (8 * torch.arange(bits, device="cuda")) & 255).to(torch.uint8).view(rows, d * bits // 8)


def _codes_of(gen, rows, d, bits):
    """Packed codes as rotated, normalised rows have them: normal entries, each the code of its nearest centroid."""
    c = torch.from_numpy(_centroids(bits, 1)).cuda()
    out, half = torch.empty((rows, d * bits // 8), dtype=torch.uint8, device="cuda"), 1 << (bits - 1)
    step = max(1, (1 << 25) // d)
    for r in range(0, rows, step):
        k = torch.bucketize(_normal(gen, min(step, rows - r), d), (c[1:] + c[:-1]) / 2)
        out[r:r + step] = _pack(torch.where(k >= half, k - half, 2 * half - 1 - k), bits)
    return out


def _prepare_product(case, gen, seed):
    n, k, m, groups = case["n"], case["k"], case["m"], case["groups"]
    s = {"case": case, "w_codes": _codes_of(gen, m, k, case["bw"]), "c_w": _centroids(case["bw"], k)}
    s["w_norms"] = (0.02 * math.sqrt(k) * (1 + 0.1 * _normal(gen, m).abs())).bfloat16()
    if case["form"] == "a16":
        s["x"] = _normal(gen, n, k).mul_(torch.exp(0.5 * _normal(gen, k))).bfloat16()
        s["perm"] = torch.randperm(k, generator=gen, device="cuda").int()
        s["signs"] = (2 * torch.randint(0, 2, (k,), generator=gen, device="cuda") - 1).to(torch.int8)
    else:
        s["x_codes"], s["c_a"] = _codes_of(gen, n, k, case["ba"]), _centroids(case["ba"], k)
        s["x_norms"] = math.sqrt(k) * torch.exp(0.2 * _normal(gen, n))
    out = DTYPES[case["out"]]
    s["bias"] = (0.5 * _normal(gen, m)).bfloat16() if case["bias"] else None
    # the gate is a slice of its layer's modulations
    s["gate"] = (0.5 * _normal(gen, groups, 6, m)).to(out)[:, 5] if case["gate"] else None
    s["residual"] = (3 * _normal(gen, n, m)).to(out) if case["residual"] else None
    s["cu"] = _ints(_bounds(case)) if case["ragged"] else None
    return s


# ------------------------------------------------------------------------------------ the passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "product": _own_product}[op](state)
    return {"norm": _plain_norm, "append": _plain_append, "product": _plain_product}[op](state)


def _own_norm(s):
    import calibration_free_w4a4_amd as orbq
    c = s["case"]
    how = dict(y=s["y"], gate=s["gate"], weight=s["weight"], scale=s["scale"], shift=s["shift"], post_weight=s["post_weight"],
               norm=c["norm"], post=c["post"] if c["residual"] and c["post"] else None, eps=EPS, cu=s["cu"])
    if not c["grad"]:
        return orbq.block_norm(s["x"], dtype=DTYPES[c["branch"]], **how)
    return tuple(orbq.block_norm_backward(s["x"], s["dh"], s["dr"], **how))


def _own_append(s):
    import calibration_free_w4a4_amd as orbq
    cache = orbq.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    rope = orbq.Rope(s["dims"], s["freqs"], s["case"]["layout"])
    q = orbq.kv_append_rope(cache, rope, s["pos"], s["q"], s["k"], s["v"], s["table"], s["start"], cu=s["cu"],
                            max_new=s["max_new"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return (q,) + tuple(orbq.kv_read(cache, s["table"], s["first"], s["cu_read"], s["total_read"], max_tokens=s["max_read"],
                                     dtype=s["k"].dtype))


def _own_product(s):
    import calibration_free_w4a4_amd as orbq
    c = s["case"]
    k, how = c["k"], dict(out_dtype=DTYPES[c["out"]], act=c["act"], bias=s["bias"], gate=s["gate"], residual=s["residual"], cu=s["cu"])
    w = orbq.Codebook.from_centroids(k, c["bw"], s["c_w"])
    if c["form"] == "a16":
        return orbq.linear_a16(s["x"], orbq.Rotation(k, 128, s["perm"], s["signs"]), s["w_codes"], s["w_norms"], w, **how)
    return orbq.lut_gemm(s["x_codes"], s["x_norms"], orbq.Codebook.from_centroids(k, c["ba"], s["c_a"]), s["w_codes"],
                         s["w_norms"], w, k, **how)


def _group_of(s, n, groups):
    """The group of each row."""
    row = torch.arange(n, device="cuda")
    return torch.searchsorted(s["cu"][1:].long(), row, right=True) if s["cu"] is not None else row // (n // groups)


def _unit(x, kind):
    """(x normalised, the factor that does it) by rows."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    f = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * f, f


def _plain_norm(s):
    c = s["case"]
    groups = c["groups"]
    g = _group_of(s, c["n"], groups)
    per = lambda v: v.float() if groups == 1 else v.float()[g]  # noqa: E731
    weight = 1.0 if s["weight"] is None else s["weight"].float()
    post_weight = 1.0 if s["post_weight"] is None else s["post_weight"].float()
    x = s["x"].float()
    u = yhat = fy = None
    if c["residual"]:
        yhat = s["y"].float()
        if c["post"]:
            yhat, fy = _unit(yhat, c["post"])
        u = yhat * post_weight
    if not c["grad"]:
        if c["residual"]:
            x = x + per(s["gate"]) * u
        h = _unit(x, c["norm"])[0] * weight * (1.0 + per(s["scale"])) + per(s["shift"])
        return x.to(s["x"].dtype), h.to(DTYPES[c["branch"]])
    rhat, f = _unit(x, c["norm"])
    dh = s["dh"].float()
    t = dh * weight * (1.0 + per(s["scale"]))
    dr = t - rhat * (t * rhat).mean(1, keepdim=True)
    if c["norm"] == "layer":
        dr = dr - t.mean(1, keepdim=True)
    dr = s["dr"].float() + f * dr
    dx = dr.to(s["x"].dtype)
    dy = None
    if c["residual"]:
        dy = dr * per(s["gate"])
        if c["post"]:
            t = dy * post_weight
            dy = t - yhat * (t * yhat).mean(1, keepdim=True)
            if c["post"] == "layer":
                dy = dy - t.mean(1, keepdim=True)
            dy = fy * dy
        dy = dy.to(s["y"].dtype)
    rows = (g == torch.arange(groups, device="cuda")[:, None]).float()      # [groups, n]: sums over the rows of each
    mod = DTYPES[c["mod"]]
    a = torch.matmul(rows, dh * rhat)
    dscale, dshift = (a * weight).to(mod), torch.matmul(rows, dh).to(mod)
    dgate = dweight = dpost = None
    if s["weight"] is not None:
        dweight = (a * (1.0 + s["scale"].float())).sum(0).to(s["weight"].dtype)
    if c["residual"]:
        b = torch.matmul(rows, dr * yhat)
        dgate = (b * post_weight).to(mod)
        if s["post_weight"] is not None:
            dpost = (b * s["gate"].float()).sum(0).to(s["post_weight"].dtype)
    return dx, dy, dgate, dweight, dscale, dshift, dpost


def _turned(x, weight, cos, sin, layout):
    y = x.float()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    r = 2 * cos.shape[-1]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if layout == "pairs" else (y[..., : r // 2], y[..., r // 2: r])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if layout == "pairs" else torch.cat((u, v), -1)
    return torch.cat((turned, y[..., r:]), -1)


def _plain_append(s):
    dims, layout = s["dims"], s["case"]["layout"]
    axis = torch.repeat_interleave(torch.arange(len(dims), device="cuda"),
                                   torch.tensor([x // 2 for x in dims], device="cuda"), output_size=sum(dims) // 2)
    angle = s["pos"][:, axis].double() * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    q = _turned(s["q"], s["q_weight"], cos, sin, layout).to(s["q"].dtype)
    k_new, v_new = _turned(s["k"], s["k_weight"], cos, sin, layout), s["v"].float()
    page = s["case"]["page"]
    start, cu, table = s["start"].long(), s["cu"].long(), s["table"].long()
    n = cu[1:] - cu[:-1]
    slots = (s["max_new"] + page - 1) // page + 1
    p = (start // page)[:, None] + torch.arange(slots, device="cuda")                       # [batch, slots]
    t = p[..., None] * page + torch.arange(page, device="cuda")                             # [batch, slots, page]
    fresh = (t >= start[:, None, None]) & (t < (start + n)[:, None, None])
    source = torch.where(fresh, cu[:-1, None, None] + t - start[:, None, None], 0)
    nobody = s["ks"].shape[0] - 1                                                           # takes what is not written
    to = torch.where(fresh.any(-1), table.gather(1, p.clamp(max=table.shape[1] - 1)), nobody)
    old = (p * page < start[:, None])[..., None]                                            # the block held tokens before
    _write(s["kc"], s["ks"], to, k_new, source, fresh, old, False)
    _write(s["vc"], s["vs"], to, v_new, source, fresh, old, True)
    i = torch.arange(s["total_read"], device="cuda")
    b = torch.searchsorted(s["cu_read"][1:].long(), i, right=True)
    at = s["first"].long()[b] + i - s["cu_read"].long()[b]
    where = table[b, at // page]
    k = s["kc"][where, :, at % page].float() * s["ks"][where][..., None]
    v = s["vc"][where, :, :, at % page].float() * s["vs"][where][..., None]
    return q, k.to(s["k"].dtype), v.to(s["k"].dtype)


def _write(codes, scales, to, x, source, fresh, old, turned):
    x = torch.where(fresh[..., None, None], x[source], 0.0).transpose(2, 3)                 # [batch, slots, heads, page, d]
    need = torch.clamp(x.abs().amax((3, 4)) * INV127, min=SCALE_FLOOR)                      # [batch, slots, heads]
    had = torch.where(old, scales[to], 0.0)
    s = torch.where(need <= had, had, torch.maximum(need, had * GROW))
    new = torch.round(x * (1.0 / s)[..., None, None]).clamp(-127, 127)
    was = codes[to].transpose(3, 4) if turned else codes[to]
    was = torch.round(was.float() * (had / s)[..., None, None])
    q = torch.where(fresh[:, :, None, :, None], new, was).to(torch.int8)
    codes[to] = q.transpose(3, 4) if turned else q
    scales[to] = s


def _values(packed, bits, centroids):
    """The bf16 centroids of packed codes (8 codes are `bits` bytes), as floats [rows, d]."""
    half = 1 << (bits - 1)
    c = torch.from_numpy(centroids).cuda().bfloat16().float()
    table = torch.cat((c[half:], c[:half].flip(0)))                # by code: magnitudes upwards, the top bit the sign
    rows = packed.shape[0]
    word = (packed.view(rows, -1, bits).long() << (8 * torch.arange(bits, device="cuda"))).sum(-1)
    return table[(word[..., None] >> (bits * torch.arange(8, device="cuda"))) & (2 * half - 1)].view(rows, -1)


def _plain_product(s):
    c = s["case"]
    w = _values(s["w_codes"], c["bw"], s["c_w"])
    if c["form"] == "a16":
        x = s["x"].float()[:, s["perm"].long()] * s["signs"].float()
        h = torch.ones((1, 1), device="cuda")
        h = functools.reduce(torch.kron, [torch.tensor([[1.0, 1.0], [1.0, -1.0]], device="cuda")] * 7, h) / math.sqrt(128)
        x = torch.matmul(x.view(c["n"], -1, 128), h).view(c["n"], -1)
    else:
        x = _values(s["x_codes"], c["ba"], s["c_a"])
    y = torch.matmul(x, w.t())
    if c["form"] != "a16":
        y = y * s["x_norms"][:, None]
    y = y * s["w_norms"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif c["act"] == "gelu_erf":
        y = 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
    if s["gate"] is not None:
        gate = s["gate"].float()
        y = y * (gate if c["groups"] == 1 else gate[_group_of(s, c["n"], c["groups"])])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


# ------------------------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        st, br, mod = SIZE[case["stream"]], SIZE[case["branch"]], SIZE[case["mod"]]
        vectors = case["groups"] * d * mod * (3 if case["residual"] else 2) * (2 if case["grad"] else 1)
        if case["grad"]:     # r, its gradients from either side, and y; the gradients of x and y
            return {"bytes": n * d * (3 * st + br + (2 * br if case["residual"] else 0)) + vectors, "flops": 30 * n * d}
        return {"bytes": n * d * (2 * st + br + (br if case["residual"] else 0)) + vectors, "flops": 12 * n * d}
    if case["op"] == "append":
        held, new = _lengths(case)
        page, size = case["page"], SIZE[case["dtype"]]
        row = 2 * case["kh"] * case["d"]
        wrote = sum(new) * (row * (size + 1) + 2 * case["qh"] * case["d"] * size)
        read = sum(h + n - h // page * page for h, n in zip(held, new)) * row * (size + 1)
        return {"bytes": wrote + read, "flops": 6 * sum(new) * (row + case["qh"] * case["d"])}
    n, k, m, out = case["n"], case["k"], case["m"], SIZE[case["out"]]
    return {"bytes": n * k * case["ba"] // 8 + m * k * case["bw"] // 8 + 2 * m + (2 * m if case["bias"] else 0)
            + n * m * out * (2 if case["residual"] else 1) + (case["groups"] * m * out if case["gate"] else 0),
            "flops": 2 * n * k * m}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "product": _exact_product}[case["op"]](s)


def _exact_norm(s):
    """The forward pass in 64 bits group by group; gradients by differentiating it."""
    c = s["case"]
    bounds = _bounds(c)
    names = ("gate", "weight", "scale", "shift", "post_weight")
    t = {a: None if s[a] is None else s[a].double() for a in names + ("x", "y")}

    def unit(x, kind):
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        return (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + EPS)

    def times(x, w):
        return x if w is None else x * w

    def branch(y, i, t):
        return times(unit(y, c["post"]) if c["post"] else y, t["post_weight"]) * t["gate"][i]

    def normed(r, i, t):
        return times(unit(r, c["norm"]), t["weight"]) * (1 + t["scale"][i]) + t["shift"][i]

    rows = [slice(a, b) for a, b in zip(bounds, bounds[1:])]
    if not c["grad"]:
        r, h = t["x"].clone(), torch.empty_like(t["x"])
        for i, at in enumerate(rows):
            if c["residual"]:
                r[at] += branch(t["y"][at], i, t)
            h[at] = normed(r[at], i, t)
        return r, h
    leaf = {a: None if t[a] is None else t[a].requires_grad_() for a in names}
    dx, dy = torch.empty_like(t["x"]), None if t["y"] is None else torch.empty_like(t["y"])
    for i, at in enumerate(rows):
        r = t["x"][at].clone().requires_grad_()
        with torch.enable_grad():
            (normed(r, i, leaf) * s["dh"][at].double()).sum().backward()
            dx[at] = r.grad + s["dr"][at].double()
            if c["residual"]:
                y = t["y"][at].clone().requires_grad_()
                (branch(y, i, leaf) * dx[at]).sum().backward()
                dy[at] = y.grad
    of = lambda a: None if leaf[a] is None else (torch.zeros_like(leaf[a]) if leaf[a].grad is None else leaf[a].grad)  # noqa: E731
    return dx, dy, of("gate"), of("weight"), of("scale"), of("shift"), of("post_weight")


def _exact_append(s):
    c = s["case"]
    page, kh, d, dims = c["page"], c["kh"], c["d"], s["dims"]
    ends = np.cumsum([0] + [x // 2 for x in dims])
    angle = torch.cat([s["pos"][:, a, None].double() * s["freqs"][ends[a]:ends[a + 1]].double() for a in range(len(dims))], 1)[:, None, :]
    i, half = torch.arange(angle.shape[-1], device="cuda"), angle.shape[-1]
    first, second = (2 * i, 2 * i + 1) if c["layout"] == "pairs" else (i, i + half)

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.double()
        r = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
        r[..., first], r[..., second] = z.real, z.imag
        return r

    start, cu, begins, cr = (s[a].tolist() for a in ("start", "cu", "first", "cu_read"))
    table = s["table"].tolist()
    out = [torch.zeros((s["total_read"], kh, d), dtype=torch.float64, device="cuda") for _ in range(2)]
    for o, x, codes, scales, tr in ((out[0], turned(s["k"], s["k_weight"]), s["kc"], s["ks"], False),
                                    (out[1], s["v"].double(), s["vc"], s["vs"], True)):
        for b in range(len(start)):
            n, begin, held = cu[b + 1] - cu[b], begins[b], start[b] - begins[b]
            new = x[cu[b]:cu[b + 1]]
            if held:                        # the block that the first new tokens join
                m = min(n, page - held)
                at = table[b][begin // page]
                q, had = codes[at].double(), scales[at].double()
                q = (q.transpose(1, 2) if tr else q)[:, :held]
                need = (new[:m].abs().amax((0, 2)) / 127).clamp(min=SCALE_FLOOR)
                v = torch.where(need <= had, had, torch.maximum(need, GROW * had))[:, None, None]
                q = torch.cat((torch.round(q * had[:, None, None] / v), torch.round(new[:m].transpose(0, 1) / v).clamp(-127, 127)), 1)
                o[cr[b]:cr[b] + held + m] = (q * v).transpose(0, 1)
                new, n = new[m:], n - m
            if n > 0:
                full = torch.nn.functional.pad(new, (0, 0, 0, 0, 0, -n % page)).view(-1, page, kh, d)
                v = (full.abs().amax((1, 3), keepdim=True) / 127).clamp(min=SCALE_FLOOR)
                o[cr[b + 1] - n:cr[b + 1]] = (torch.round(full / v).clamp(-127, 127) * v).reshape(-1, kh, d)[:n]
    return turned(s["q"], s["q_weight"]), out[0], out[1]


def _exact_product(s):
    c = s["case"]

    def values(packed, bits, centroids):
        """Bit by bit: bit j of code i is bit (i bits + j) of its row."""
        c = torch.from_numpy(centroids).cuda().bfloat16().double()
        b = (packed[..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
        b = b.view(packed.shape[0], -1, bits)
        half = 1 << (bits - 1)
        rank = sum((b[..., j].long() << j for j in range(bits - 1)), torch.zeros_like(b[..., 0], dtype=torch.int64))
        return torch.where(b[..., bits - 1] == 1, -c[half + rank], c[half + rank])

    w = values(s["w_codes"], c["bw"], s["c_w"]) * s["w_norms"].double()[:, None]
    out, bounds = torch.empty((c["n"], c["m"]), dtype=torch.float64, device="cuda"), _bounds(c)
    if c["form"] == "a16":
        x = s["x"].double()[:, s["perm"].long()] * s["signs"].double()
        x = x.view(c["n"], -1, 128)
        i = torch.arange(128, device="cuda")
        odd = sum(((i[:, None] & i) >> j) & 1 for j in range(7)) & 1
        x = (x @ ((1 - 2 * odd).double() / math.sqrt(128))).reshape(c["n"], -1)
    for i in range(c["groups"]):
        for r in range(bounds[i], bounds[i + 1], 4096):
            at = slice(r, min(r + 4096, bounds[i + 1]))
            a = x[at] if c["form"] == "a16" else values(s["x_codes"][at], c["ba"], s["c_a"]) * s["x_norms"][at].double()[:, None]
            y = a @ w.t()
            if s["bias"] is not None:
                y += s["bias"].double()
            if c["act"] == "gelu_tanh":
                y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
            elif c["act"] == "gelu_erf":
                y = y * torch.special.ndtr(y)
            if s["gate"] is not None:
                y *= s["gate"][i].double()
            out[at] = y if s["residual"] is None else y + s["residual"][at].double()
    return out
