"""Pins of the attention sublayer's float64 oracle (CPU): closed forms, and the
backward against central differences of the forward."""

import numpy as np
import pytest

from oracle import attn_oracle as A


def _angles(n, rot, rng):
    a = rng.uniform(-3, 3, (n, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot,dh", [(0, 8), (4, 8), (8, 8)])
def test_rotation_keeps_norms_and_turns_pairs(adjacent, rot, dh):
    rng = np.random.default_rng(0)
    cs = _angles(5, rot, rng)
    R = A.rotation(cs, np.array([4, 0, 2]), rot, dh, adjacent)
    assert np.allclose(R @ R.transpose(0, 2, 1), np.eye(dh))
    z = rng.standard_normal(dh)
    y = R[0] @ z
    assert np.allclose(y[rot:], z[rot:])
    if rot:
        a, b = (0, 1) if adjacent else (0, rot // 2)
        turned = (z[a] + 1j * z[b]) * (cs[4, 0] + 1j * cs[4, rot // 2])
        assert np.allclose([y[a], y[b]], [turned.real, turned.imag])


def test_norm_rope_has_unit_rms():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 8)) * 100
    R = A.rotation(_angles(3, 8, rng), np.arange(3), 8, 8, False)
    y = A.norm_rope(x, np.ones(8), R, 0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0)


@pytest.mark.parametrize("adjacent", [False, True])
def test_backward_matches_central_differences(adjacent):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 2, 8)), 1 + 0.3 * rng.standard_normal(8)
    g = rng.standard_normal(x.shape)
    R = A.rotation(_angles(3, 4, rng), np.arange(3), 4, 8, adjacent)
    dx, dw = A.norm_rope_bwd(g, x, w, R, 1e-3)
    f = lambda x, w: (g * A.norm_rope(x, w, R, 1e-3)).sum()     # noqa: E731
    h = 1e-6
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(8):
        d = np.zeros(8)
        d[i] = h
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((6, 1, 4)), rng.standard_normal((6, 1, 4))
    # equal scores: the mean of the values a row sees
    o, lse, _, _ = A.attention(np.zeros((2, 2, 4)), k, v, 1.0)
    assert np.allclose(o[1, 0], v[:, 0].mean(0)) and np.allclose(lse[1], np.log(6))
    assert np.allclose(o[0, 1], v[:5, 0].mean(0))
    # a window of one: the row's own value
    o, lse, _, _ = A.attention(rng.standard_normal((2, 2, 4)), k, v, 1.0, window=1)
    assert np.allclose(o[:, 0], v[4:, 0]) and np.allclose(o[:, 1], v[4:, 0])
    # more new tokens than cached ones: the first rows see nothing
    o, lse, _, _ = A.attention(rng.standard_normal((8, 2, 4)), k, v, 1.0)
    assert np.all(o[:2] == 0) and np.all(lse[:2] == -np.inf) and np.all(np.isfinite(lse[2:]))
    # a large cap changes nothing
    q = rng.standard_normal((2, 2, 4))
    assert np.allclose(A.attention(q, k, v, 0.5)[0], A.attention(q, k, v, 0.5, softcap=1e6)[0])
