"""The block_norm oracle: its norms by their defining properties, its gradients against central differences."""
import numpy as np
import pytest

from oracle import block_norm as ob


def test_unit():
    rng = np.random.default_rng(0)
    v = rng.standard_normal(500) * 3 + 7
    z, _ = ob.unit(v, "layer", 0.0)
    assert abs(z.mean()) < 1e-12 and abs((z * z).mean() - 1) < 1e-12
    z, _ = ob.unit(v, "rms", 0.0)
    assert abs((z * z).mean() - 1) < 1e-12 and np.allclose(z / v, z[0] / v[0])
    assert np.array_equal(ob.unit(np.zeros(4), "rms", 1e-6)[0], np.zeros(4))


@pytest.mark.parametrize("norm", ["layer", "rms", None])
@pytest.mark.parametrize("post", ["layer", "rms", None])
@pytest.mark.parametrize("cu", [None, [1, 3, 3, 7]])
def test_gradients_by_differences(norm, post, cu):
    rng = np.random.default_rng(1)
    n, d, groups, eps = 9, 6, 3, 1e-3
    v = {a: rng.standard_normal(s) for a, s in dict(x=(n, d), y=(n, d), gate=(groups, d), scale=(groups, d), shift=(groups, d),
                                                    weight=(d,), post_weight=(d,)).items()}
    dr, dh = rng.standard_normal((n, d)), rng.standard_normal((n, d))

    def run(v):
        r = ob.stream(v["x"], v["y"], v["gate"], v["post_weight"] if post else None, post, eps, groups, cu)
        rows = [i for g in ob.groups_of(n, groups, cu) for i in g]
        loss = (dr[rows] * r[rows]).sum()
        if norm is not None:
            loss += (dh[rows] * ob.normed(r, v["weight"], v["scale"], v["shift"], norm, eps, groups, cu)[rows]).sum()
        return loss, r

    got = ob.gradients(run(v)[1], dr, dh, v["y"], v["gate"], v["weight"] if norm else None, v["scale"] if norm else None,
                       v["post_weight"] if post else None, norm, post, eps, eps, groups, cu)
    step = 1e-5
    for name in v:
        if (norm is None and name in ("scale", "shift", "weight")) or (post is None and name == "post_weight"):
            continue
        for at in np.ndindex(v[name].shape):
            up, down = ({**v, name: v[name].copy()} for _ in range(2))
            up[name][at] += step
            down[name][at] -= step
            want = (run(up)[0] - run(down)[0]) / (2 * step)
            assert abs(got[name][at] - want) < 1e-6 * (1 + abs(want)), (name, at)
