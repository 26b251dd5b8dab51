"""Pins of the block-norm oracle: the formulas by loops, and every gradient
against central differences in FP64."""

import math

import numpy as np
import pytest

from oracle import norm as on

KINDS = [("rms", "rms"), ("layer", "layer"), (None, "rms"), ("rms", "layer"), ("layer", None)]


def test_forward_by_loops():
    rng = np.random.default_rng(0)
    M, D, seg, eps, alpha = 5, 6, 2, 1e-3, 0.7
    h, b = rng.standard_normal((M, D)), rng.standard_normal((M, D))
    gate, scale, shift = (rng.standard_normal((3, D)) for _ in range(3))
    ho = on.residual(h, b, gate, alpha, eps, "rms", seg)
    n = on.modulated(ho, scale, shift, eps, "layer", seg)
    for m in range(M):
        s = m // seg
        r = 1 / math.sqrt(sum(v * v for v in b[m]) / D + eps)
        want = [alpha * h[m, i] + gate[s, i] * b[m, i] * r for i in range(D)]
        assert np.allclose(ho[m], want, rtol=1e-13)
        mean = sum(want) / D
        r = 1 / math.sqrt(sum((v - mean) ** 2 for v in want) / D + eps)
        assert np.allclose(n[m], [(want[i] - mean) * r * (1 + scale[s, i]) + shift[s, i] for i in range(D)], rtol=1e-12)


@pytest.mark.parametrize("post,pre", KINDS)
def test_gradients_against_differences(post, pre):
    rng = np.random.default_rng(7)
    M, D, seg, eps, alpha = 5, 8, 2, 1e-3, 0.7
    a = {k: rng.standard_normal((M, D)) for k in ("h", "b")}
    a |= {k: rng.standard_normal((3, D)) for k in ("gate", "scale", "shift")}
    dn, dho = rng.standard_normal((M, D)), rng.standard_normal((M, D))

    def loss(v):
        ho = on.residual(v["h"], v["b"], v["gate"], alpha, eps, post, seg)
        total = (dho * ho).sum()
        return total if pre is None else total + (dn * on.modulated(ho, v["scale"], v["shift"], eps, pre, seg)).sum()

    ho = on.residual(a["h"], a["b"], a["gate"], alpha, eps, post, seg)
    got = dict(zip(("h", "b", "gate", "scale", "shift"),
                   on.backward(dn if pre else None, dho, ho, a["b"], a["gate"], a["scale"] if pre else None, alpha, eps,
                               post, pre, seg)))
    for name, g in got.items():
        if g is None:
            assert pre is None and name in ("scale", "shift")
            continue
        num = np.zeros_like(a[name])
        for i in np.ndindex(num.shape):
            step = np.zeros_like(num)
            step[i] = 1e-5
            num[i] = (loss({**a, name: a[name] + step}) - loss({**a, name: a[name] - step})) / 2e-5
        assert np.abs(num - g).max() < 1e-8, name


def test_no_block_output():
    rng = np.random.default_rng(3)
    h, dn = rng.standard_normal((4, 8)), rng.standard_normal((4, 8))
    dh, db, dgate, dscale, dshift = on.backward(dn, None, h, None, None, None, 1.0, 1e-6, None, "rms", 4)
    assert db is None and dgate is None and dscale.shape == dshift.shape == (1, 8)
    assert np.abs((dh * h).sum(1)).max() < 1e-5  # N is homogeneous of degree 0 (up to eps)
