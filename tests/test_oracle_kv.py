"""Pins of the key/value cache oracle: closed forms, worked cases, the code order."""
import numpy as np
import pytest

from oracle import msq_kv as O


def test_worked_block():
    """Scale 2/127 and the half-to-even ties of a hand-made block."""
    c = O.Cache(2, 1, 64, 32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :4] = [254, -254, 3, 5]          # scale 2: 127, -127, 1.5 -> 2, 2.5 -> 2
    c.write(x, x, np.array([[1]]), [0], [0, 2])
    assert c.scale["k"][1, 0] == 2 and c.scale["k"][0, 0] == 0
    assert list(c.codes["k"][1, 0, 0, :5]) == [127, -127, 2, 2, 0]
    y = np.zeros((1, 1, 64), np.float32)
    y[0, 0, 0] = 508                          # the scale grows to 4: 127 -> 63.5 -> 64, 2 -> 1
    c.write(y, y, np.array([[1]]), [2], [0, 1])
    assert c.scale["k"][1, 0] == 4
    assert list(c.codes["k"][1, 0, 0, :4]) == [64, -64, 1, 1]
    assert c.codes["k"][1, 0, 2, 0] == 127
    z = np.full((1, 1, 64), 8, np.float32)    # a smaller token keeps the scale
    c.write(z, z, np.array([[1]]), [3], [0, 1])
    assert c.scale["k"][1, 0] == 4 and c.codes["k"][1, 0, 3, 0] == 2


@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (256, 32)])
def test_round_trip_within_half_a_step(D, P):
    rng = np.random.default_rng(D)
    c = O.Cache(3, 2, D, P)
    x = rng.normal(size=(2 * P, 2, D)).astype(np.float32)
    c.write(x, 3 * x, np.array([[2, 0]]), [0], [0, 2 * P])
    for name, f in (("k", 1), ("v", 3)):
        back = c.values(name, np.array([2, 0]), 0, 2 * P)
        step = c.scale[name][np.repeat([2, 0], P)][:, :, None]
        assert (np.abs(back - f * x) <= step * (0.5 + 1e-4)).all()


def test_special_values():
    x = np.array([np.nan, np.inf, -np.inf, 1.0, 0.0], np.float32)
    assert list(O.code_of(x, np.float32(1 / 127))) == [0, 127, -127, 127, 0]
    assert list(O.code_of(x, np.float32(0))) == [0] * 5


@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (128, 256), (256, 128)])
def test_code_orders_are_permutations(D, P):
    t, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    for f in (O.key_byte, O.value_byte):
        assert np.array_equal(np.sort(f(t, d, D).ravel()), np.arange(P * D))


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(5, 1, 8))
    q, k = np.zeros((2, 2, 8)), rng.normal(size=(5, 1, 8))
    out, lse = O.attention(q, k, v, O.sees(5, 2), 1.0)[:2]   # equal weights
    assert np.allclose(out[0, 0], v[:4, 0].mean(0)) and np.allclose(out[1, 1], v[:, 0].mean(0))
    assert np.allclose(lse, np.log([[4, 4], [5, 5]]))
    out, lse = O.attention(q, k, v, O.sees(5, 2, window=1), 1.0)[:2]
    assert np.allclose(out[:, 0], v[3:, 0])
    q = np.zeros((7, 2, 8))                                    # rows before the first token
    out, lse = O.attention(q, k, v, O.sees(5, 7), 1.0)[:2]
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
