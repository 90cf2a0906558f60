"""The many-row form whose tiles are laid out in f16 before (k_turn, k_turned): enough row tiles read them, on one
stream and on many, split and whole.  That a call takes this form is seen in the workspace, whose first tile holds the
first stream's codes."""
import numpy as np
import pytest

from tests.gpu_common import log, torch_mod
from tests.test_gpu_attention import ints, orbq, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = {128: 256, 256: 128}          # rows of a workgroup


def first_tile_is_turned(ws, c, table, page, d, first):
    """The workspace begins with 64 keys [d / 8][64][8] in f16, from token `first` (a multiple of 64) on."""
    torch = torch_mod()
    got = ws[:2 * 64 * d].view(torch.float16).view(d // 8, 64, 8).permute(1, 0, 2).reshape(64, d)
    for t in range(64):
        pg = int(table[0, (first + t) // page])
        if pg >= 0 and not torch.equal(got[t], c.k_codes[pg, 0, (first + t) % page].half()):
            return False
    return True


@pytest.mark.parametrize("d,heads,kv_heads,page,lens,new,split,kw", [
    # whole: as many row tiles as compute units, or a full last round
    (128, 32, 16, 64, [1200, 1100], [1000, 1000], False, dict(block=1)),
    (128, 32, 32, 32, [2060], [2000], False, dict()),
    (256, 32, 16, 64, [700, 600], [500, 500], False, dict(block=37, window=450)),
    # split: two sequences, heads that share a cache head, blocks that are absent, frames, windows, no mask
    (128, 6, 2, 64, [900, 1000], [700, 650], True, dict(block=37, absent=((0, 3), (1, 0), (1, 9)))),
    (128, 4, 4, 128, [2500, 1900], [2000, 1900], True, dict(block=1)),
    (128, 3, 1, 16, [1400], [1300], True, dict(block=300, window=1000, absent=((0, 20),))),
    (128, 4, 1, 64, [6000], [470], True, dict(pads=(2, 8))),
    (128, 2, 2, 32, [6100], [2000], True, dict(block=156)),
    (256, 4, 2, 64, [900, 800, 470], [500, 480, 470], True, dict(block=1, absent=((2, 1), (0, 8)))),
    (256, 2, 1, 128, [5000], [500], True, dict(block=0)),
    (256, 1, 1, 16, [2000], [1100], True, dict(block=50, window=1000)),
    # scores and scales of every size
    (128, 2, 1, 64, [1300], [1000], True, dict(block=1, peak=20.0)),
    (128, 2, 1, 64, [1300], [1000], True, dict(block=1, vary=8.0, scale=-0.3)),
    (256, 2, 1, 64, [1000], [500], True, dict(vary=8.0))])
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_tiles_turned_before(orbq, name, d, heads, kv_heads, page, lens, new, split, kw):  # noqa: F811
    torch = torch_mod()
    log(f"turned {name} d={d} heads {heads}/{kv_heads} page={page} {lens} {new} {kw}")
    kw = dict(kw)
    block, window = kw.get("block", 0), kw.get("window", 0)
    most = max(new)
    assert -(-most * (heads // kv_heads) // ROWS[d]) >= 8        # row tiles
    c, q, table, o = run_attention(orbq, name, d, page, heads, kv_heads, lens, new, **kw)
    cu = ints(np.concatenate([[0], np.cumsum(new)]))
    args = dict(cu=cu, max_new=most, causal_block=block, window=window, scale=kw.get("scale"))
    need = orbq.kv_attention_workspace_bytes(c, len(lens), sum(new), most, heads, table.shape[1] * page, block, window)
    ws = torch.full((need,), 0x55, dtype=torch.uint8, device="cuda")
    first = lens[0] - new[0]                                     # position of the first query
    hi = min(lens[0], (first // block + 1) * block) if block else lens[0]
    first = max(0, hi - window) // 64 * 64 if window else 0
    again = orbq.kv_attention(c, q, ints(table), ints(lens), workspace=ws, **args)
    assert torch.equal(again, o.contiguous())
    assert first_tile_is_turned(ws, c, table, page, d, first)
    tiles = -(-table.shape[1] * page // 64) if not window else -(-(window + most + block) // 64) + 1
    tiles = min(tiles, -(-table.shape[1] * page // 64) + (1 if window else 0))
    parts = need - len(lens) * kv_heads * tiles * (256 * d + 64)
    assert (parts > 0) == split and parts % ((d + 2) * 4) == 0, parts
    # a guess at the lengths forbids it, and gives the same up to rounding
    ws.fill_(0x55)
    other = orbq.kv_attention(c, q, ints(table), ints(lens), max_len=max(lens) // 2, workspace=ws, **args)
    assert not first_tile_is_turned(ws, c, table, page, d, first)
    assert (other.float() - o.float()).abs().max().item() <= 2.0 ** -7 * o.float().abs().max().item()


@pytest.mark.parametrize("d,heads,kv_heads,lens,new,window", [
    (128, 2, 1, [2700], [1100], 1500), (256, 2, 1, [2000], [600], 900)])
def test_turned_blocks_before_the_window_may_hold_anything(orbq, d, heads, kv_heads, lens, new, window):  # noqa: F811
    """As for the other forms: blocks that no query sees, some in the first window's first tile, hold scales that are no numbers."""
    torch = torch_mod()
    log(f"turned, before the window d={d}")
    page = 16
    first = lens[0] - new[0] + 1 - window
    assert first % 64 >= 16
    c, q, table, o = run_attention(orbq, "bf16", d, page, heads, kv_heads, lens, new, block=1, window=window)
    hidden = torch.from_numpy(table[0, :first // page].astype(np.int64)).cuda()
    need = orbq.kv_attention_workspace_bytes(c, 1, new[0], new[0], heads, table.shape[1] * page, 1, window)
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    for k, v in (("inf", "inf"), ("-inf", "nan"), ("nan", "-inf")):
        c.k_scales[hidden] = float(k)
        c.v_scales[hidden] = float(v)
        ws.fill_(0x55)
        assert torch.equal(orbq.kv_attention(c, q, ints(table), ints(lens), causal_block=1, window=window, workspace=ws), o), (k, v)
        assert first_tile_is_turned(ws, c, table, page, d, first // 64 * 64)


@pytest.mark.parametrize("d", [128, 256])
def test_turned_scores_of_the_largest_magnitude(orbq, d):  # noqa: F811
    """Scores down to -2^25 in the form that reads turned tiles."""
    torch = torch_mod()
    page, heads, n, new = 64, 2, 300, 2000 if d == 128 else 1000
    c = orbq.KVCache.create(8, heads, d, page)
    rng = np.random.default_rng(d)
    table = ints(np.arange(5)[None])
    k = np.zeros((n, heads, d), np.float32)
    k[:, :, 0] = -rng.uniform(90, 127, (n, 1))
    v = rng.standard_normal((n, heads, d)).astype(np.float32)
    orbq.kv_append(c, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), table, ints([0]))
    rk, rv = orbq.kv_read(c, table, ints([0]), None, n, dtype=torch.float32)
    q = torch.zeros((new, heads, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0 ** 18
    ws = torch.full((orbq.kv_attention_workspace_bytes(c, 1, new, new, heads, 320),), 0x55, dtype=torch.uint8, device="cuda")
    o = orbq.kv_attention(c, q, table, ints([n]), scale=1.0, workspace=ws)
    assert first_tile_is_turned(ws, c, table.cpu().numpy(), page, d, 0)
    for h in range(heads):
        top = rk[:, h, 0].max()
        mean = rv[rk[:, h, 0] == top, h].double().mean(0)
        err = (o[:, h].double() - mean).abs()
        assert bool((err <= 2.0 ** -8 * mean.abs() + 2.0 ** -10 * rv.abs().max()).all())
