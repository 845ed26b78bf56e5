"""CPU pins of the oracle's position rotation and single-token attention."""
import numpy as np
import pytest

from oracle.attention import causal_attention
from oracle.decode import attend_one
from oracle.rope import rotate


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32])
def test_rotation_is_a_complex_product_and_depends_on_distances_only(interleaved, rot):
    rng = np.random.default_rng(3)
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    x = rng.normal(size=(5, 2, 32))
    pos = np.array([0, 1, 17, 2**20 + 3, -9])
    y = rotate(x, pos, f, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., rot:], x[..., rot:])
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None] * f)[:, None]
    assert np.allclose(y[..., a] + 1j * y[..., b], z, atol=1e-9)
    assert np.allclose(rotate(y, pos, f, interleaved, back=True), x, atol=1e-9)
    # q at m and k at n meet at an angle of m - n
    q, k = rng.normal(size=(2, 1, 1, 32))
    near = [np.sum(rotate(q, [p + 7], f, interleaved) * rotate(k, [p], f, interleaved))
            for p in (0, 100, 12345)]
    assert np.allclose(near, near[0], atol=1e-8)


def test_rotation_back_is_the_gradient_by_differences():
    rng = np.random.default_rng(5)
    f, pos = np.array([1.0, 0.3, 0.01, 0.002] * 2), np.array([3, 250])
    x, dy, w = rng.normal(size=(3, 2, 3, 16))
    eps = 1e-5
    rise = np.sum(dy * (rotate(x + eps * w, pos, f) - rotate(x - eps * w, pos, f))) / (2 * eps)
    assert np.isclose(rise, np.sum(rotate(dy, pos, f, back=True) * w), rtol=1e-8)


def test_single_token_attention_is_the_last_row_of_full_attention():
    rng = np.random.default_rng(7)
    L, Hq, Hkv, d = 13, 6, 2, 8
    q, k, v = (rng.normal(size=(L, h, d)) for h in (Hq, Hkv, Hkv))
    o, lse = causal_attention(q, k, v, 0.4)[:2]
    for n in (1, 5, L):
        got_o, got_lse, spread = attend_one(q[n - 1], k[:n], v[:n], 0.4)
        assert np.allclose(got_o, o[n - 1]) and np.allclose(got_lse, lse[:, n - 1])
        assert (spread >= np.abs(got_o) - 1e-12).all()
    o, lse, _ = attend_one(q[0], k[:0], v[:0], 0.4)
    assert not o.any() and np.isneginf(lse).all()
