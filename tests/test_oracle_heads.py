"""Pins of the float64 definitions of the rotation and of the linear attention with a decay for each
head: closed forms, sums over pairs of tokens, and central differences."""
import numpy as np
import pytest

from oracle import heads as H

EPS = 1e-6


def difference(f, x, d, h=1e-5):
    """Central difference of the number f(x) along d (error h^2 of a cubic term)."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotation_is_a_product_of_complex_numbers(neighbours):
    rng = np.random.default_rng(0)
    x, freqs = rng.normal(size=(5, 2, 10)), rng.normal(size=3)
    pos = rng.integers(-50, 50, size=(5, 2))
    a = H.angles(pos, freqs, [1, 2])
    np.testing.assert_array_equal(a[:, 0], pos[:, 0] * freqs[0])
    np.testing.assert_array_equal(a[:, 1:], pos[:, 1:] * freqs[1:])
    y = H.rope_fwd(x, None, a, neighbours, False, EPS)
    one, two = (slice(0, 6, 2), slice(1, 6, 2)) if neighbours else (slice(0, 3), slice(3, 6))
    z = (x[..., one] + 1j * x[..., two]) * np.exp(1j * a)[:, None]
    np.testing.assert_allclose(y[..., one], z.real, atol=1e-14)
    np.testing.assert_allclose(y[..., two], z.imag, atol=1e-14)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])


def test_rotated_products_see_distances_alone():
    rng = np.random.default_rng(1)
    q, k, w = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8)), rng.normal(size=8)
    freqs = rng.normal(size=4)

    def at(x, p):
        return H.rope_fwd(x, w, H.angles(np.array([[p]]), freqs, [4]), False, True, EPS)

    near = (at(q, 7) * at(k, 3)).sum()
    np.testing.assert_allclose((at(q, 1007) * at(k, 1003)).sum(), near, rtol=1e-10)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
def test_rope_gradients(norm, neighbours):
    rng = np.random.default_rng(2)
    x, w, dy = rng.normal(size=(4, 3, 7)), rng.normal(size=7), rng.normal(size=(4, 3, 7))
    a = rng.normal(size=(4, 2)) * 5
    dx, dw = H.rope_bwd(x, w, a, neighbours, norm, EPS, dy)
    d = rng.normal(size=x.shape)
    got = difference(lambda x: (H.rope_fwd(x, w, a, neighbours, norm, EPS) * dy).sum(), x, d)
    np.testing.assert_allclose(got, (dx * d).sum(), rtol=1e-7)
    if norm:
        d = rng.normal(size=w.shape)
        got = difference(lambda w: (H.rope_fwd(x, w, a, neighbours, norm, EPS) * dy).sum(), w, d)
        np.testing.assert_allclose(got, (dw * d).sum(), rtol=1e-7)


def draw(L=9, Hq=4, Hkv=2, dk=3, dv=5, seed=3):
    rng = np.random.default_rng(seed)
    return (rng.normal(size=(L, Hq, dk)), rng.normal(size=(L, Hkv, dk)), rng.normal(size=(L, Hkv, dv)),
            -rng.uniform(0.01, 0.7, size=Hkv), rng.normal(size=(Hkv, dk, dv)), 0.7)


def test_decay_is_a_sum_over_pairs():
    q, k, v, l, s0, scale = draw()
    o, last = H.decay_fwd(q, k, v, l, s0, scale)
    L = len(q)
    for h in range(4):
        for i in range(L):
            want = np.exp(l[h // 2] * (i + 1)) * q[i, h] @ s0[h // 2]
            for j in range(i + 1):
                want = want + np.exp(l[h // 2] * (i - j)) * (q[i, h] @ k[j, h // 2]) * v[j, h // 2]
            np.testing.assert_allclose(o[i, h], scale * want, rtol=1e-12)
    want = np.exp(l * L)[:, None, None] * s0 + sum(
        np.exp(l * (L - 1 - j))[:, None, None] * k[j][:, :, None] * v[j][:, None] for j in range(L))
    np.testing.assert_allclose(last, want, rtol=1e-12)


def test_decay_of_minus_infinity_sees_the_token_itself():
    q, k, v, _, s0, scale = draw(Hq=2)
    o, last = H.decay_fwd(q, k, v, np.full(2, -np.inf), s0, scale)
    np.testing.assert_allclose(o, scale * (q * k).sum(-1, keepdims=True) * v, rtol=1e-12)
    np.testing.assert_allclose(last, k[-1][:, :, None] * v[-1][:, None], rtol=1e-12)


def test_decay_gradients():
    q, k, v, l, s0, scale = draw()
    rng = np.random.default_rng(4)
    do, ds = rng.normal(size=(9, 4, 5)), rng.normal(size=s0.shape)

    def f(q, k, v, s0):
        o, last = H.decay_fwd(q, k, v, l, s0, scale)
        return (o * do).sum() + (last * ds).sum()

    args = [q, k, v, s0]
    for i, g in enumerate(H.decay_bwd(q, k, v, l, s0, scale, do, ds)):
        d = rng.normal(size=args[i].shape)
        got = difference(lambda x: f(*args[:i], x, *args[i + 1:]), args[i], d)
        np.testing.assert_allclose(got, (g * d).sum(), rtol=1e-7)


def test_absolute_bounds_the_values():
    q, k, v, l, s0, scale = draw()
    rng = np.random.default_rng(5)
    do, ds = rng.normal(size=(9, 4, 5)), rng.normal(size=s0.shape)
    for a, b in zip(H.decay_fwd(q, k, v, l, s0, scale), H.decay_fwd(q, k, v, l, s0, scale, True)):
        assert (np.abs(a) <= b * (1 + 1e-12)).all()
    for a, b in zip(H.decay_bwd(q, k, v, l, s0, scale, do, ds), H.decay_bwd(q, k, v, l, s0, scale, do, ds, True)):
        assert (np.abs(a) <= b * (1 + 1e-12)).all()
    x, w, ang = rng.normal(size=(4, 3, 7)), rng.normal(size=7), rng.normal(size=(4, 2))
    for near in (False, True):
        y, m = (H.rope_fwd(x, w, ang, near, True, EPS, absolute=t) for t in (False, True))
        assert (np.abs(y) <= np.abs(m) * (1 + 1e-12)).all()
        for a, b in zip(H.rope_bwd(x, w, ang, near, True, EPS, x * 2), H.rope_bwd(x, w, ang, near, True, EPS, x * 2, True)):
            assert (np.abs(a) <= b * (1 + 1e-12)).all()
