"""The fp64 forms of norm, rotation, the 4-bit format and attention, pinned to
values and identities that need no other implementation."""

import numpy as np
import pytest

from oracle import heads as OH


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 3, 16))
    f = 10.0 ** -np.arange(4)
    pos = np.array([0, 1, 7, 1000, 123456])
    y, _ = OH.turn(x, None, pos, f, 0.0, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # a product of two heads depends on the distance of their positions alone
    a, _ = OH.turn(x, None, pos + 40, f, 0.0, interleaved)
    b, _ = OH.turn(x[::-1], None, pos[::-1] + 40, f, 0.0, interleaved)
    c, _ = OH.turn(x[::-1], None, pos[::-1], f, 0.0, interleaved)
    assert np.allclose((a * b[::-1]).sum(-1), (y * c[::-1]).sum(-1))
    # one pair by hand
    ia, ib = (2, 3) if interleaved else (1, 5)
    assert np.isclose(y[2, 0, ia], x[2, 0, ia] * np.cos(0.7) - x[2, 0, ib] * np.sin(0.7))
    assert np.isclose(y[2, 0, ib], x[2, 0, ib] * np.cos(0.7) + x[2, 0, ia] * np.sin(0.7))


def test_norm():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, _ = OH.turn(x, np.array([1.0, 2.0, 1.0, 1.0]), None, None, 0.0, False)
    assert np.allclose(y, [[[1.2, 3.2, 0.0, 0.0]]])
    assert np.allclose(OH.turn(x, np.ones(4), None, None, 18.75, False)[0], x / 5.0)


def test_scales_and_levels():
    x = np.zeros((6, 32))
    x[:5, 0] = [7.0, 7.0001, 3.5, -14.0, 1e-30]
    assert OH.scale_exponent(x)[:, 0].tolist()[:4] == [0, 1, -1, 1]
    assert OH.scale_exponent(x)[5, 0] == -126
    for top in (1e-30, 0.3, 5.0, 7.5, 1e30):
        e = OH.scale_exponent(np.full((1, 32), top))[0, 0]
        assert top <= 7 * 2.0 ** e and top > 7 * 2.0 ** (e - 1)
    a = np.array([0, .25, .26, .75, 1.25, 1.26, 1.75, 2.5, 2.6, 3.5, 5.0, 5.1, 6.9, 7.0, -.25, -2.6] * 2)
    want = [0, 0, .5, 1, 1, 1.5, 2, 2, 3, 4, 4, 6, 6, 6, 0, -3]
    assert OH.nearest(a, np.zeros(1))[:16].tolist() == want
    # codes: one byte holds two channels, the even one below
    v = OH.values(np.array([[0x21, 0xF9] + [0] * 14], np.uint8), np.array([[128]], np.uint8))
    assert v[0, :4].tolist() == [1.0, 2.0, -1.0, -12.0]
    assert np.isnan(OH.values(np.zeros((1, 16), np.uint8), np.array([[255]], np.uint8))).all()


def test_attention():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((6, 2, 8)), g.standard_normal((6, 2, 8))
    see = np.tril(np.ones((3, 6), bool), 3)
    see[1] = False
    o, lse, size = OH.attend(q, k, v, see, 0.3)
    assert (o[1] == 0).all() and (lse[1] == -np.inf).all() and (size >= np.abs(o) - 1e-12).all()
    x = 0.3 * (k[:4, 1] @ q[0, 3])
    assert np.isclose(lse[0, 3], np.log(np.exp(x).sum()))
    assert np.allclose(o[0, 3], np.exp(x) @ v[:4, 1] / np.exp(x).sum())
