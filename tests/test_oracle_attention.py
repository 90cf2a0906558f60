"""Pins of the attention-side oracle (CPU): closed forms and identities, independent of the GPU path."""
import numpy as np
import pytest

from oracle import attention as oa


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_is_orthogonal_and_relative(layout):
    rng = np.random.default_rng(0)
    dims, d = (8, 6, 6), 24
    freqs = rng.uniform(0.01, 1.0, 10).astype(np.float32)
    x, y = rng.standard_normal((2, 1, 1, d))
    p, q, shift = rng.uniform(-50, 50, (3, 1, 3)).astype(np.float32)
    px, qy = oa.rope(x, dims, freqs, p, layout), oa.rope(y, dims, freqs, q, layout)
    assert np.allclose(np.linalg.norm(px), np.linalg.norm(x))
    assert np.array_equal(px[..., 20:], x[..., 20:])                        # the rest passes through
    assert np.allclose(oa.rope(px, dims, freqs, p, layout, inverse=True), x)
    moved = (oa.rope(x, dims, freqs, p.astype(np.float64) + shift, layout) *
             oa.rope(y, dims, freqs, q.astype(np.float64) + shift, layout)).sum()
    assert np.allclose(moved, (px * qy).sum())                               # only differences of positions count


def test_rope_axes_one_at_a_time():
    freqs = np.array([0.5, 0.25, 2.0], np.float32)
    x = np.zeros((1, 1, 6)); x[..., 0::2] = 1.0
    y = oa.rope(x, (2, 2, 2), freqs, np.array([[3.0, 0.0, 0.0]], np.float32), "pairs")
    assert np.allclose(y[0, 0], [np.cos(1.5), np.sin(1.5), 1, 0, 1, 0])


def test_append_block_rules():
    x = np.array([[127.0, -1.0], [0.5, 1.5]], np.float32)
    c, s = oa.append_block(np.zeros((4, 2), np.int8), np.float32(np.nan), 0, x)
    assert abs(float(s) - 1.0) < 1e-6 and c[0, 0] == 127 and c[0, 1] == -1
    c2, s2 = oa.append_block(c, s, 2, np.array([[3.0, np.nan]], np.float32))
    assert s2 == s and c2[2].tolist() == [3, 0] and np.array_equal(c2[:2], c[:2])
    c3, s3 = oa.append_block(c, s, 2, np.array([[130.0, -np.inf]], np.float32))
    assert s3 == np.float32(1.25) * s and c3[0, 0] == 102 and c3[2].tolist() == [104, -127]
    c4, s4 = oa.append_block(c, s, 0, np.zeros((2, 2), np.float32))
    assert s4 == np.float32(2.0 ** -64) and not c4[:2].any()


def test_growing_again_and_again_costs_at_most_two_and_a_half_steps():
    rng = np.random.default_rng(1)
    x = rng.uniform(-1, 1, (64, 8)).astype(np.float32) * np.float32(1.02) ** np.arange(64, dtype=np.float32)[:, None]
    codes, s = np.zeros((64, 8), np.int8), np.float32(0)
    for t in range(64):
        codes, s = oa.append_block(codes, s, t, x[t:t + 1])
    assert np.abs(codes * np.float64(s) - x).max() <= 2.5 * s


def test_attention_masks_and_closed_forms():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((5, 2, 4)), rng.standard_normal((9, 1, 4)), rng.standard_normal((9, 1, 4))
    o, lse, _ = oa.attention(np.zeros_like(q), k, v, 0, 0, 1.0)              # equal weights
    assert np.allclose(o, v.mean(0)) and np.allclose(lse, np.log(9))
    o, lse, _ = oa.attention(q, k, v, 1, 1, 0.5)                            # one key a query: its own
    assert np.allclose(o, v[4:]) and np.allclose(lse[:, 0], 0.5 * (q[:, 0] * k[4:, 0]).sum(-1))
    o, lse, _ = oa.attention(q, k[:3], v[:3], 1, 0, 0.5)                    # queries before the first token
    assert not o[:2].any() and np.all(np.isneginf(lse[:2])) and np.allclose(o[2], v[0])
    lo, hi = oa.visible(10, 6, 4, 0)
    assert hi.tolist() == [8, 8, 8, 8, 10, 10] and not lo.any()
    assert oa.visible(10, 6, 4, 3)[0].tolist() == [5, 5, 5, 5, 7, 7]
    o, _, _ = oa.attention(q, k[:0], v[:0], 0, 0, 1.0)
    assert not o.any()
