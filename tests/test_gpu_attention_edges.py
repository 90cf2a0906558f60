"""Calls at the edges of what the attention-side operators take: bounds below the counts, positions outside the
sequence, bounds far above the work."""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_common import log, torch_mod
from tests.test_gpu_attention import cache_of, check_attention, dev, host, ints, orbq, table_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,heads,kv_heads,lens,new,most,block,window", [
    (64, 2, 2, [200, 90], [7, 3], 2, 1, 0), (128, 4, 2, [200, 90], [9, 3], 4, 1, 37), (256, 2, 1, [200, 5], [7, 9], 3, 16, 0),
    (128, 4, 4, [30000], [7], 2, 1, 0), (64, 4, 2, [700, 300], [400, 299], 90, 1, 0), (64, 2, 2, [700], [400], 90, 0, 70),
    (128, 4, 2, [700, 300], [400, 310], 90, 50, 130), (256, 2, 2, [700], [333], 70, 1, 33),
    (128, 2, 1, [1500], [1400], 1100, 1, 0), (128, 2, 1, [1900], [1600], 1100, 37, 900), (256, 2, 1, [900, 500], [700, 600], 500, 1, 450)])
def test_a_bound_below_the_counts_moves_no_position(orbq, d, heads, kv_heads, lens, new, most, block, window):  # noqa: F811
    """Query i of a sequence's n stands at len - n + i, whether or not max_new leaves the last ones out."""
    torch = torch_mod()
    log(f"bound {most} of {new} d={d} heads {heads}/{kv_heads} {lens} block {block} window {window}")
    rng = np.random.default_rng(d + most)
    page = 64
    pages = sum(-(-n // page) for n in lens) + 2
    table = table_of(rng, pages, lens, page)
    c = cache_of(orbq, rng, pages, kv_heads, d, page)
    c.k_scales.copy_(torch.from_numpy((np.exp(rng.standard_normal((pages, kv_heads))) / 40).astype(np.float32)))
    total, cu = sum(new), np.concatenate([[0], np.cumsum(new)])
    q, q64 = dev(rng.standard_normal((total, heads, d)), "bf16")
    out, lse = torch.full_like(q, 7.0), torch.full((total, heads), 7.0, device="cuda")
    orbq.kv_attention(c, q, ints(table), ints(lens), cu=ints(cu), max_new=most, causal_block=block, window=window, out=out,
                      lse=lse)
    kc, vc, ks, vs = host(c)
    for b, n in enumerate(lens):
        k, v = oa.kv_tokens(kc, ks, table[b], n, False), oa.kv_tokens(vc, vs, table[b], n, True)
        want = oa.attention(q64[cu[b]:cu[b + 1]], k, v, block, window, d ** -0.5)
        m = min(most, new[b])
        check_attention(out[cu[b]:cu[b] + m], lse[cu[b]:cu[b] + m], tuple(x[:m] for x in want), d, "bf16", n)
        assert bool((out[cu[b] + m:cu[b + 1]] == 7.0).all()) and bool((lse[cu[b] + m:cu[b + 1]] == 7.0).all())


@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
def test_tokens_before_the_first_read_as_zero(orbq, name, d, page):  # noqa: F811
    """Every row of the output is written: zero at negative positions, the tokens behind them as they are held."""
    torch = torch_mod()
    log(f"read before token 0 {name} d={d} page={page}")
    rng = np.random.default_rng(page)
    heads, n = 3, 2 * page + 9
    first = [-5, -page, -3 * page - 1, -2 ** 31, 0]
    pages = 5 * 3
    table = np.arange(pages, dtype=np.int32).reshape(5, 3)
    c = cache_of(orbq, rng, pages, heads, d, page)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    out = [torch.full((5 * n, heads, d), float("nan"), dtype=dt, device="cuda") for _ in range(2)]
    orbq.kv_read(c, ints(table), ints(first), None, 5 * n, out=out)
    kc, vc, ks, vs = host(c)
    for o, codes, scales, turned in ((out[0], kc, ks, False), (out[1], vc, vs, True)):
        for b, f in enumerate(first):
            zeros = min(n, -f)
            held = oa.kv_tokens(codes, scales, table[b], n, turned)[:n - zeros].astype(np.float32)
            want = np.concatenate([np.zeros((zeros, heads, d), np.float32), held])
            assert torch.equal(o[b * n:(b + 1) * n].cpu(), torch.from_numpy(want).to(dt)), b


@pytest.mark.parametrize("d,page", [(64, 16), (256, 128)])
def test_a_bound_far_above_the_work(orbq, d, page):  # noqa: F811
    """The largest bound a caller may give for a call of few tokens: the same bits as with their number."""
    torch = torch_mod()
    log(f"bound 2^30 d={d} page={page}")
    rng = np.random.default_rng(d)
    heads, held, new = 2, [0, 3, 700], [3, 0, 2]
    total, lens = sum(new), [a + b for a, b in zip(held, new)]
    table = table_of(rng, 100, lens, page, extra=1)
    a, b = (cache_of(orbq, np.random.default_rng(1), 100, heads, d, page) for _ in range(2))
    x, _ = dev(rng.standard_normal((total, heads, d)), "bf16")
    args = dict(cu=ints(np.concatenate([[0], np.cumsum(new)])))
    most = 2 ** 30
    orbq.kv_append(a, x, x, ints(table), ints(held), max_new=max(new), **args)
    orbq.kv_append(b, x, x, ints(table), ints(held), max_new=most, **args)
    for g, w in zip(host(b), host(a)):
        assert np.array_equal(g, w)
    want = orbq.kv_read(a, ints(table), ints(held), args["cu"], total, max_tokens=max(new))
    got = orbq.kv_read(a, ints(table), ints(held), args["cu"], total, max_tokens=most)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    want = orbq.kv_attention(a, x, ints(table), ints(lens), max_new=total, causal_block=1, **args)
    assert torch.equal(orbq.kv_attention(a, x, ints(table), ints(lens), max_new=most, causal_block=1, **args), want)


@pytest.mark.parametrize("new", [1, 70])
def test_no_expected_length(orbq, new):  # noqa: F811
    """max_len 0 says nothing, as in C: the call is split as the table asks for, and finds its workspace."""
    torch = torch_mod()
    rng = np.random.default_rng(new)
    c = cache_of(orbq, rng, 300, 1, 128, 128)
    table, lens = ints(np.arange(300)[None]), ints([38001])
    q, _ = dev(rng.standard_normal((new, 1, 128)), "bf16")
    assert torch.equal(orbq.kv_attention(c, q, table, lens, max_len=0), orbq.kv_attention(c, q, table, lens))


@pytest.mark.parametrize("d,batch,heads,kv_heads,each", [(64, 1024, 256, 64, 8), (128, 1024, 256, 64, 8)])
def test_more_row_tiles_than_one_launch_takes(orbq, d, batch, heads, kv_heads, each):  # noqa: F811
    """Many short sequences whose bound nobody gave: 2^24 (2^23) row tiles of 256 (512) threads, almost all of them empty."""
    torch = torch_mod()
    log(f"loose bound d={d} batch={batch} heads {heads}/{kv_heads}")
    gen = torch.Generator(device="cuda").manual_seed(d)
    total = batch * each
    c = orbq.KVCache.create(batch, kv_heads, d, 16)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(-127, 128, t.shape, generator=gen, device="cuda", dtype=torch.int8))
    for t in (c.k_scales, c.v_scales):
        t.fill_(1 / 40)
    table = torch.randperm(batch, generator=gen, device="cuda").int()[:, None]
    lens = torch.randint(each, 17, (batch,), generator=gen, device="cuda", dtype=torch.int32)
    cu = ints(np.arange(batch + 1) * each)
    q = torch.randn((total, heads, d), generator=gen, device="cuda").bfloat16()
    want = orbq.kv_attention(c, q, table, lens, cu=cu, max_new=each, causal_block=1)
    got = orbq.kv_attention(c, q, table, lens, cu=cu, causal_block=1)
    assert -(-total * (heads // kv_heads) // (128 if d == 64 else 256)) * batch * kv_heads * (256 if d == 64 else 512) >= 2 ** 32
    assert (got.float() - want.float()).abs().max().item() <= 2.0 ** -7 * want.float().abs().max().item()


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_is_in_the_autograd_graph(orbq, name, layout):  # noqa: F811
    """Its gradients are rope_backward's, whichever inputs ask for them and however the incoming ones lie."""
    torch = torch_mod()
    log(f"autograd {name} {layout}")
    rng = np.random.default_rng(2)
    r = orbq.Rope.create((16, 24, 24), layout=layout)
    p, _ = dev(rng.integers(0, 60, (31, 3)))
    q, k, gq, gk = (dev(rng.standard_normal((31, h, 72)), name)[0] for h in (6, 2, 6, 2))
    want = orbq.rope(r, p, q, k)
    back = orbq.rope_backward(r, p, gq, gk)
    q.requires_grad_(True)
    k.requires_grad_(True)
    y = orbq.rope(r, p, q, k)
    assert all(torch.equal(a, b) and a.requires_grad for a, b in zip(y, want))
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (q, k), (gq, gk)), back))
    # one output's gradient alone, one input alone, one tensor alone
    y = orbq.rope(r, p, q, k)
    dq, dk = torch.autograd.grad(y[1], (q, k), gk, allow_unused=True)
    assert dq is None and torch.equal(dk, back[1])
    y = orbq.rope(r, p, q.detach(), k)
    assert torch.equal(torch.autograd.grad(y, k, (gq, gk))[0], back[1])
    assert torch.equal(torch.autograd.grad(orbq.rope(r, p, q), q, gq)[0], back[0])
    # an expanded gradient, whose last dimension has no stride
    ones = torch.ones_like(gq)
    assert torch.equal(torch.autograd.grad(orbq.rope(r, p, q).sum(), q)[0], orbq.rope_backward(r, p, ones))
    # the gradient's gradient is the turn again
    v = gq.clone().requires_grad_(True)
    dq, = torch.autograd.grad(orbq.rope(r, p, q), q, v, create_graph=True)
    assert torch.equal(torch.autograd.grad(dq, v, gq)[0], orbq.rope(r, p, gq))
    # nothing is recorded where nothing is asked for
    with torch.no_grad():
        assert not orbq.rope(r, p, q).requires_grad
    out = torch.empty_like(gq)
    assert orbq.rope(r, p, q, out=out) is out and not out.requires_grad and torch.equal(out, want[0])


def test_a_gradient_through_the_cache_is_refused(orbq):  # noqa: F811
    """Not lost without a word: the output is in the graph, and a backward pass that reaches it raises."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    c = cache_of(orbq, rng, 4, 2, 64, 16)
    table, lens = ints([[0, 1, 3]]), ints([40])
    q, _ = dev(rng.standard_normal((5, 4, 64)), "bf16")
    want = orbq.kv_attention(c, q, table, lens, causal_block=1)
    q.requires_grad_(True)
    o = orbq.kv_attention(c, q, table, lens, causal_block=1)
    assert torch.equal(o, want) and o.requires_grad
    with pytest.raises(orbq.OrbqError):
        o.sum().backward()
    with torch.no_grad():
        assert not orbq.kv_attention(c, q, table, lens, causal_block=1).requires_grad
    out = torch.empty_like(want)
    assert orbq.kv_attention(c, q, table, lens, causal_block=1, out=out) is out and not out.requires_grad and torch.equal(out, want)


@pytest.mark.parametrize("d,batch,heads,kv_heads,new,n,unbound", [
    (64, 64, 16, 16, 1, 12000, False), (128, 64, 16, 16, 1, 12000, False), (256, 64, 16, 16, 1, 12000, False),
    (64, 32, 1280, 32, 1, 12000, False), (128, 32, 1280, 32, 1, 12000, False),
    (64, 1, 64, 1, 1536, 60000, False), (128, 1, 64, 1, 1024, 60000, True), (128, 1, 64, 1, 1024, 60000, False),
    (256, 1, 64, 1, 512, 60000, True), (256, 1, 64, 1, 512, 60000, False)])
def test_many_small_weights_beside_a_large_one(orbq, d, batch, heads, kv_heads, new, n, unbound):  # noqa: F811
    """One key in the first tile of each wave takes nearly all the weight, with a value of zero; all others have 2^-25.4 of it
    and a value of one.  A weight is rounded by 2^-28 of the largest at most, so n of them lose n 2^-28 of it."""
    torch = torch_mod()
    page = 64
    pages = -(-n // page)
    few = new * heads // kv_heads <= 64
    tiles = 4 if few else 1                  # the first tiles of the waves; a workgroup of the few-row form has four of them
    log(f"small weights d={d} {'few' if few else 'many'} unbound {unbound}")
    c = orbq.KVCache.create(pages, kv_heads, d, page)
    c.k_codes.zero_()
    c.v_codes.fill_(127)
    c.k_codes[:tiles, :, 0, 0] = 127
    c.v_codes[:tiles, :, :, 0] = 0
    c.k_scales.fill_(1 / 127)
    c.v_scales.fill_(1 / 127)
    table = ints(np.tile(np.arange(pages), (batch, 1)))
    q = torch.zeros((batch * new, heads, d), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 16.0
    bits = 25.4
    ks = float(np.float32(1 / 127)) * 127
    scale = float(np.float32(bits * math.log(2) / (16 * ks)))
    w = math.exp(-scale * 16 * ks)
    want = (n - tiles) * w / (tiles + (n - tiles) * w)
    # nothing is split: the workspace has room for turned tiles alone
    assert orbq.kv_attention_workspace_bytes(c, batch, batch * new, new, heads, pages * page) == (0 if few or d == 64 else
                                                                                                   pages * (256 * d + 64))
    o = orbq.kv_attention(c, q, table, ints([n] * batch), scale=scale, max_len=n if unbound else None).double()
    tol = (n - tiles) * 2.0 ** -28 / tiles + 2.0 ** -9 * want + 2.0 ** -25
    assert tol < want / 2
    assert (o - want).abs().max().item() <= tol, ((o - want).abs().max().item(), want, tol)
