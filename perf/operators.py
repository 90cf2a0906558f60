"""Cases of the attention-side operators: rotary positions with several axes, the 8-bit paged
key/value cache (quantised as it is written, and read back), and attention over that cache.

`own = False` computes them in their plain form (elementary torch operations in 32 bits, rounded
once at the end); `own = True` calls the framework.  Sizes: the video layers' 21 x 30 x 52 latent
tokens (1560 a frame) and width 1536 as 12 heads of 128, image layers of 512 text and 64 x 64 image
tokens; batched and long token-by-token serving sizes are generic.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
SCALE_FLOOR = 2.0 ** -64      # the least scale of a block of the cache
GROW = 1.25                   # a block's scale that has to grow grows at least by this factor
INV127 = float(np.float32(1.0) / np.float32(127.0))


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of a token-by-token decoder, its q and k in one call: latency
        {"name": "rope_token", "op": "rope", "text": 1, "t": 0, "h": 0, "w": 0, "qh": 12, "kh": 12, "d": 128,
         "dims": "44,42,42", "layout": "pairs", "dtype": "bf16", "grad": False},
        # q and k of a whole video clip, 21 frames of 30 x 52 latent tokens
        {"name": "rope_video", "op": "rope", "text": 0, "t": 21, "h": 30, "w": 52, "qh": 12, "kh": 12, "d": 128,
         "dims": "44,42,42", "layout": "pairs", "dtype": "bf16", "grad": False},
        # gradient of q and k of an image layer in training, 509 text and 64 x 64 image tokens, 32 bits,
        # fewer k than q heads and the split-half order of pairs
        {"name": "rope_image_grad", "op": "rope", "text": 509, "t": 1, "h": 64, "w": 64, "qh": 24, "kh": 8, "d": 128,
         "dims": "16,56,56", "layout": "halves", "dtype": "f32", "grad": True},
        # one token appended to each of 48 running sequences, and their last blocks read back: latency
        {"name": "cache_step", "op": "cache", "batch": 48, "new": 1, "ragged": False, "held": 8000, "kh": 8, "d": 128,
         "page": 64, "dtype": "bf16"},
        # three frames of a video written behind the 18 held ones (and some text tokens), and read back
        {"name": "cache_frames", "op": "cache", "batch": 1, "new": 4680, "ragged": False, "held": 28117, "kh": 12,
         "d": 128, "page": 64, "dtype": "bf16"},
        # prompts of a ragged batch written into short blocks, narrow heads
        {"name": "cache_prompts", "op": "cache", "batch": 7, "new": 5000, "ragged": True, "held": 0, "kh": 4, "d": 64,
         "page": 16, "dtype": "f16"},
        # one query token over a short cache: latency
        {"name": "attn_step", "op": "attn", "batch": 1, "new": 1, "ragged": False, "len": 777, "qh": 12, "kh": 12,
         "d": 128, "page": 64, "dtype": "bf16", "block": 1, "window": 0},
        # one query token for each of 48 sequences of ragged lengths, four query heads a k/v head
        {"name": "attn_batch_step", "op": "attn", "batch": 48, "new": 1, "ragged": True, "len": 16384, "qh": 32,
         "kh": 8, "d": 128, "page": 64, "dtype": "bf16", "block": 1, "window": 0},
        # four query tokens (drafted ahead) over one long cache, eight query heads a k/v head
        {"name": "attn_long_step", "op": "attn", "batch": 1, "new": 4, "ragged": False, "len": 262157, "qh": 64,
         "kh": 8, "d": 64, "page": 128, "dtype": "f16", "block": 1, "window": 0},
        # the next three frames of a video attend to all 21, frame by frame: each sees its own and earlier frames
        {"name": "attn_frames", "op": "attn", "batch": 1, "new": 4680, "ragged": False, "len": 32760, "qh": 12,
         "kh": 12, "d": 128, "page": 64, "dtype": "bf16", "block": 1560, "window": 0},
        # ragged prompts behind cached prefixes, causal with a window, short blocks, narrow heads
        {"name": "attn_prompts", "op": "attn", "batch": 7, "new": 3001, "ragged": True, "len": 7001, "qh": 16, "kh": 4,
         "d": 64, "page": 16, "dtype": "f16", "block": 1, "window": 1024},
        # image and text tokens that all see each other, wide heads
        {"name": "attn_image", "op": "attn", "batch": 2, "new": 4605, "ragged": False, "len": 4605, "qh": 8, "kh": 4,
         "d": 256, "page": 64, "dtype": "bf16", "block": 0, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "rope":
        kh = rng.choice([1, 2, 4, 8, 12])
        d, dims = rng.choice([(128, "44,42,42"), (128, "16,56,56"), (64, "16,24,24"), (256, "64,64,64"), (128, "32,48,48")])
        frame = rng.random() < 0.5
        return {"op": "rope", "text": _log(rng, 1, 4096), "t": _log(rng, 1, 16) if frame else 0,
                "h": rng.randint(1, 41) if frame else 0, "w": rng.randint(1, 43) if frame else 0,
                "qh": kh * rng.choice([1, 2, 3]) if kh < 12 else 12, "kh": kh, "d": d, "dims": dims,
                "layout": rng.choice(["pairs", "halves"]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "grad": rng.random() < 0.5}
    kh, d, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "cache":
        batch = _log(rng, 1, 64)
        return {"op": "cache", "batch": batch, "new": _log(rng, 1, 4096 // batch), "ragged": rng.random() < 0.5,
                "held": rng.choice([0, _log(rng, 1, 4096)]), "kh": kh, "d": d, "page": page, "dtype": dtype}
    group = rng.choice([1, 2, 4, 7])
    if rng.random() < 0.5:      # a few query tokens over a cache of up to 200 MB
        batch, new = _log(rng, 1, 64), rng.choice([1, 1, 1, rng.randint(2, 9)])
        n = new + _log(rng, 1, min(200000, 10 ** 8 // (batch * kh * d)))
    else:                       # many, with no more than 6 * 10^8 scores or 6 * 10^11 operations
        batch = _log(rng, 1, 6)
        new = min(_log(rng, 10, 3000), int(math.sqrt(1.5e11 / (batch * kh * group * d))))
        n = new + _log(rng, 1, max(1, min(6000, 6 * 10 ** 8 // (batch * kh * group * new) - new)))
    return {"op": "attn", "batch": batch, "new": new, "ragged": rng.random() < 0.5, "len": n, "qh": kh * group, "kh": kh,
            "d": d, "page": page, "dtype": dtype, "block": rng.choice([0, 1, 1, rng.randint(2, 1600)]),
            "window": rng.choice([0, 0, _log(rng, 1, 4096)])}


def _lengths(case):
    """(tokens before the call, new tokens) of each sequence: part of the case, not of the seed."""
    rng = random.Random("%(batch)d %(new)d %(d)d %(page)d" % case)
    n, h = case["new"], case["held"] if case["op"] == "cache" else case["len"] - case["new"]
    new = [rng.randint(1, n) if case["ragged"] else n for _ in range(case["batch"])]
    # sequences of a batch are never all as long as the longest
    return [rng.randint(h // 8, h) if case["batch"] > 1 else h for _ in range(case["batch"])], new


def _tokens(case):
    return case["text"] + case["t"] * case["h"] * case["w"]


# ------------------------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, gen)
    return _prepare_cache(case, gen, seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _prepare_rope(case, gen):
    n, d, dt = _tokens(case), case["d"], DTYPES[case["dtype"]]
    dims = [int(x) for x in case["dims"].split(",")]
    # text tokens count up on all axes alike; then the grid of frames, rows and columns
    pos = torch.empty((n, len(dims)), device="cuda")
    pos[: case["text"]] = (torch.arange(case["text"], device="cuda") % 256)[:, None].float()
    t, h, w = (torch.arange(case[a], device="cuda", dtype=torch.float32) for a in "thw")
    pos[case["text"]:] = torch.cartesian_prod(t, h, w).reshape(-1, 3)
    pos += torch.randint(1, 64, (1,), generator=gen, device="cuda")     # a segment that starts somewhere
    freqs = np.concatenate([10000.0 ** (-np.arange(0, k, 2) / k) for k in dims])
    return {"case": case, "dims": dims, "pos": pos, "freqs": torch.from_numpy(freqs).float().cuda(),
            "q": _normal(gen, n, case["qh"], d).to(dt), "k": _normal(gen, n, case["kh"], d).to(dt)}


def _prepare_cache(case, gen, seed):
    held, new = _lengths(case)
    batch, page, kh, d, dt = case["batch"], case["page"], case["kh"], case["d"], DTYPES[case["dtype"]]
    lens = [a + b for a, b in zip(held, new)]
    per = [(x + page - 1) // page for x in lens]
    pages = sum(per) + 3                      # the last one is nobody's
    order = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed), dtype=torch.int64)
    table = torch.zeros((batch, max(per)), dtype=torch.int32)
    table[torch.arange(max(per)) < torch.tensor(per)[:, None]] = order[: sum(per)].int()
    table = table.cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = ints([0] + np.cumsum(new).tolist())
    # blocks of full 8-bit range with scales as blocks of heavy-tailed keys and values have them;
    # blocks that no sequence holds are as the allocator left them
    codes = lambda: torch.round(_normal(gen, pages, kh, page * d) * 30).clamp_(-127, 127).to(torch.int8)  # noqa: E731
    scales = lambda s: (s / 30) * torch.exp(0.3 * _normal(gen, pages, kh))  # noqa: E731
    kc, vc = codes().view(pages, kh, page, d), codes().view(pages, kh, d, page)
    ks, vs = scales(1.0), scales(1.0)
    nobody = order[sum(per):].cuda()
    ks[nobody] = vs[nobody] = float("nan")
    st = {"case": case, "table": table, "cu": cu, "max_new": max(new), "kc": kc, "vc": vc, "ks": ks, "vs": vs}
    total = sum(new)
    if case["op"] == "attn":
        return {**st, "lens": ints(lens), "q": (1.5 * _normal(gen, total, case["qh"], d)).to(dt)}
    first = [h // page * page for h in held]  # what is read back: the new tokens and the block they joined
    read = [x - f for x, f in zip(lens, first)]
    heavy = lambda: (_normal(gen, total, kh, d) * torch.exp(0.3 * _normal(gen, total, kh, 1))).to(dt)  # noqa: E731
    return {**st, "start": ints(held), "k": heavy(), "v": heavy(), "first": ints(first),
            "cu_read": ints([0] + np.cumsum(read).tolist()), "total_read": sum(read), "max_read": max(read)}


# ------------------------------------------------------------------------------------ the passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "cache": _own_cache, "attn": _own_attn}[op](state)
    return {"rope": _plain_rope, "cache": _plain_cache, "attn": _plain_attn}[op](state)


def _own_rope(s):
    import calibration_free_w4a4_amd as orbq
    rope = orbq.Rope(s["dims"], s["freqs"], s["case"]["layout"])
    if s["case"]["grad"]:
        return orbq.rope_backward(rope, s["pos"], s["q"], s["k"])
    return orbq.rope(rope, s["pos"], s["q"], s["k"])


def _own_cache(s):
    import calibration_free_w4a4_amd as orbq
    cache = orbq.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    orbq.kv_append(cache, s["k"], s["v"], s["table"], s["start"], cu=s["cu"], max_new=s["max_new"])
    return orbq.kv_read(cache, s["table"], s["first"], s["cu_read"], s["total_read"], max_tokens=s["max_read"],
                        dtype=s["k"].dtype)


def _own_attn(s):
    import calibration_free_w4a4_amd as orbq
    cache = orbq.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return orbq.kv_attention(cache, s["q"], s["table"], s["lens"], cu=s["cu"], max_new=s["max_new"],
                             causal_block=s["case"]["block"], window=s["case"]["window"])


def _plain_rope(s):
    c, dims = s["case"], s["dims"]
    axis = torch.repeat_interleave(torch.arange(len(dims), device="cuda"),
                                   torch.tensor([x // 2 for x in dims], device="cuda"), output_size=sum(dims) // 2)
    angle = s["pos"][:, axis] * s["freqs"]
    cos, sin = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :]
    sin = -sin if c["grad"] else sin
    return _rotate(s["q"], cos, sin, c["layout"]), _rotate(s["k"], cos, sin, c["layout"])


def _rotate(x, cos, sin, layout):
    r = 2 * cos.shape[-1]
    y = x.to(cos.dtype)
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if layout == "pairs" else (y[..., : r // 2], y[..., r // 2: r])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if layout == "pairs" else torch.cat((u, v), -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _plain_cache(s):
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
    _write(s["kc"], s["ks"], to, s["k"], source, fresh, old, False)
    _write(s["vc"], s["vs"], to, s["v"], source, fresh, old, True)
    i = torch.arange(s["total_read"], device="cuda")
    b = torch.searchsorted(s["cu_read"][1:].long(), i, right=True)
    at = s["first"].long()[b] + i - s["cu_read"].long()[b]
    where = table[b, at // page]
    k = s["kc"][where, :, at % page].float() * s["ks"][where][..., None]
    v = s["vc"][where, :, :, at % page].float() * s["vs"][where][..., None]
    return k.to(s["k"].dtype), v.to(s["k"].dtype)


def _write(codes, scales, to, x, source, fresh, old, turned):
    x = torch.where(fresh[..., None, None], x[source].float(), 0.0).transpose(2, 3)         # [batch, slots, heads, page, d]
    need = torch.clamp(x.abs().amax((3, 4)) * INV127, min=SCALE_FLOOR)                      # [batch, slots, heads]
    had = torch.where(old, scales[to], 0.0)
    s = torch.where(need <= had, had, torch.maximum(need, had * GROW))
    new = torch.round(x * (1.0 / s)[..., None, None]).clamp(-127, 127)
    was = codes[to].transpose(3, 4) if turned else codes[to]
    was = torch.round(was.float() * (had / s)[..., None, None])
    q = torch.where(fresh[:, :, None, :, None], new, was).to(torch.int8)
    codes[to] = q.transpose(3, 4) if turned else q
    scales[to] = s


def _limits(case, lens, n, most):
    """First and one past the last visible key of each query [batch, most]."""
    pos = (lens - n)[:, None] + torch.arange(most, device="cuda")
    hi = lens[:, None].expand_as(pos)
    if case["block"]:
        hi = torch.minimum(hi, torch.where(pos < 0, 0, (pos // case["block"] + 1) * case["block"]))
    return (torch.clamp(hi - case["window"], min=0) if case["window"] else torch.zeros_like(hi)), hi


def _plain_attn(s):
    c, table, cu, lens = s["case"], s["table"].long(), s["cu"].long(), s["lens"].long()
    batch, kh, d, most = c["batch"], c["kh"], c["d"], s["max_new"]
    g, total, n = c["qh"] // kh, s["q"].shape[0], cu[1:] - cu[:-1]
    keys = table.shape[1] * c["page"]
    k = (s["kc"][table].float() * s["ks"][table][..., None, None]).transpose(1, 2).reshape(batch, kh, keys, d)
    v = (s["vc"][table].float() * s["vs"][table][..., None, None]).permute(0, 2, 1, 4, 3).reshape(batch, kh, keys, d)
    j = torch.arange(keys, device="cuda")
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    source = (cu[:-1, None] + torch.arange(most, device="cuda")).clamp(max=total - 1)       # [batch, most]
    q = s["q"].float()[source].view(batch, most, kh, g, d).permute(0, 2, 3, 1, 4).reshape(batch, kh, g * most, d)
    lo, hi = _limits(c, lens, n, most)
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, None]                       # [batch, 1, 1, most, keys]
    a = torch.matmul(q, k.transpose(2, 3)).view(batch, kh, g, most, keys)
    a = a.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen, float("-inf"))
    a = a.sub_(a.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    l = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(batch, kh, g * most, keys), v).view(batch, kh, g, most, d)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 3, 1, 2, 4).reshape(batch, most, c["qh"], d)
    b = torch.searchsorted(cu[1:], torch.arange(total, device="cuda"), right=True)
    return o[b, torch.arange(total, device="cuda") - cu[b]].to(s["q"].dtype)


# ------------------------------------------------------------------------------------ what a pass needs
def work(case):
    size, d = SIZE[case["dtype"]], case["d"]
    if case["op"] == "rope":
        n, r = _tokens(case), sum(int(x) for x in case["dims"].split(","))
        heads = case["qh"] + case["kh"]
        return {"bytes": 2 * n * heads * d * size + n * 12 + 2 * r, "flops": 3 * n * heads * r}
    held, new = _lengths(case)
    if case["op"] == "cache":
        page = case["page"]
        row = 2 * case["kh"] * d
        wrote = sum(new) * row * (size + 1)
        read = sum(h + n - h // page * page for h, n in zip(held, new)) * row * (size + 1)
        return {"bytes": wrote + read, "flops": 3 * (wrote + read) / (size + 1)}
    pairs, keys = 0, 0
    for h, n in zip(held, new):
        pos = h + np.arange(n, dtype=np.int64)
        hi = np.minimum(h + n, (pos // case["block"] + 1) * case["block"]) if case["block"] else np.full(n, h + n)
        lo = np.maximum(hi - case["window"], 0) if case["window"] else np.zeros_like(hi)
        pairs += int((hi - lo).sum())
        keys += int(hi.max() - lo.min())
    return {"bytes": 2 * keys * case["kh"] * (d + 4 / case["page"]) + 2 * sum(new) * case["qh"] * d * size,
            "flops": 4 * pairs * case["qh"] * d}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    def of_rope(s):
        c, out = s["case"], []
        bounds = np.cumsum([0] + [x // 2 for x in s["dims"]])
        angle = torch.cat([s["pos"][:, a, None].double() * s["freqs"][bounds[a]:bounds[a + 1]].double()
                           for a in range(len(s["dims"]))], 1)
        angle = (-angle if c["grad"] else angle)[:, None, :]
        half = angle.shape[-1]
        for x in (s["q"], s["k"]):
            y = x.double()
            r = y.clone()
            i = torch.arange(half, device="cuda")
            first, second = (2 * i, 2 * i + 1) if c["layout"] == "pairs" else (i, i + half)
            z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
            r[..., first], r[..., second] = z.real, z.imag
            out.append(r)
        return tuple(out)

    def of_cache(s):
        page, kh, d = s["case"]["page"], s["case"]["kh"], s["case"]["d"]
        start, cu, first, cr = (s[a].tolist() for a in ("start", "cu", "first", "cu_read"))
        table = s["table"].tolist()
        out = [torch.zeros((s["total_read"], kh, d), dtype=torch.float64, device="cuda") for _ in range(2)]
        for o, x, codes, scales, turned in ((out[0], s["k"], s["kc"], s["ks"], False), (out[1], s["v"], s["vc"], s["vs"], True)):
            for b in range(len(start)):
                n = cu[b + 1] - cu[b]
                begin, held = first[b], start[b] - first[b]
                new = x[cu[b]:cu[b + 1]].double()
                if held:                        # the block that the first new tokens join
                    m = min(n, page - held)
                    at = table[b][begin // page]
                    q = codes[at].double()
                    q = (q.transpose(1, 2) if turned else q)[:, :held]
                    had = scales[at].double()
                    need = (new[:m].abs().amax((0, 2)) / 127).clamp(min=SCALE_FLOOR)
                    v = torch.where(need <= had, had, torch.maximum(need, GROW * had))[:, None, None]
                    q = torch.round(q * had[:, None, None] / v)
                    q = torch.cat((q, torch.round(new[:m].transpose(0, 1) / v).clamp(-127, 127)), 1)
                    o[cr[b]:cr[b] + held + m] = (q * v).transpose(0, 1)
                    new, begin, n = new[m:], begin + page, n - m
                if n > 0:
                    full = torch.nn.functional.pad(new, (0, 0, 0, 0, 0, -n % page)).view(-1, page, kh, d)
                    v = (full.abs().amax((1, 3), keepdim=True) / 127).clamp(min=SCALE_FLOOR)
                    got = (torch.round(full / v).clamp(-127, 127) * v).reshape(-1, kh, d)[:n]
                    o[cr[b + 1] - n:cr[b + 1]] = got
        return tuple(out)

    def of_attn(s):
        c, lens, cu = s["case"], s["lens"].tolist(), s["cu"].tolist()
        g, d, page = c["qh"] // c["kh"], c["d"], c["page"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            m = cu[b + 1] - cu[b]
            pos = torch.arange(n - m, n, device="cuda")
            hi = torch.full_like(pos, n)
            if c["block"]:
                hi = torch.clamp((torch.div(pos, c["block"], rounding_mode="floor") + 1) * c["block"], max=n)
                hi[pos < 0] = 0
            lo = torch.clamp(hi - c["window"], min=0) if c["window"] else torch.zeros_like(hi)
            j = torch.arange(n, device="cuda")
            at = s["table"][b, : (n + page - 1) // page].long()
            for h in range(c["kh"]):
                k = (s["kc"][at, h].double() * s["ks"][at, h].double()[:, None, None]).reshape(-1, d)[:n]
                v = (s["vc"][at, h].double() * s["vs"][at, h].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:n]
                for r in range(0, m, 2048):
                    seen = (j >= lo[r:r + 2048, None]) & (j < hi[r:r + 2048, None])
                    some = seen.any(1)[:, None, None]
                    q = s["q"][cu[b] + r:min(cu[b] + r + 2048, cu[b + 1]), h * g:(h + 1) * g].double()
                    a = (q @ k.t()) / math.sqrt(d)
                    a = torch.softmax(a.masked_fill(~seen[:, None, :], float("-inf")), -1)
                    out[cu[b] + r:cu[b] + r + q.shape[0], h * g:(h + 1) * g] = torch.where(some, a @ v, 0.0)
        return out

    s = prepare(case, seed)
    return {"rope": of_rope, "cache": of_cache, "attn": of_attn}[case["op"]](s)
