"""Pins of the oracles of rotary positions and drafted tokens: closed forms, worked cases, and that
verification by chance gives every token the target's probability."""
import numpy as np
import pytest

from oracle import msq_draft as T
from oracle import msq_rotary as R


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    freq = 10000.0 ** (-np.arange(8) / 8)
    x = rng.normal(size=(5, 2, 24)).astype(np.float32)
    at = np.array([0, 1, -3, 1000, 123456])
    y = R.rotate(x, at, freq, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
    want = R.rotate64(x, at, freq, interleaved)
    size = np.abs(x).max() * 2
    assert np.abs(y - want).max() <= size * 2.0 ** -22
    # a quarter turn: (a, b) -> (-b, a)
    z = R.rotate(x[:1], [1], np.full(8, np.pi / 2), interleaved)
    lo, hi = R.pairs(16, interleaved)
    assert np.allclose(z[..., lo], -x[:1][..., hi], atol=1e-6) and np.allclose(z[..., hi], x[:1][..., lo], atol=1e-6)
    # lengths stay, amplitude scales, the inverse comes back
    assert np.allclose(np.square(want).sum(-1), np.square(x.astype(float)).sum(-1))
    assert np.allclose(R.rotate64(want, -at, freq, interleaved), x)
    assert np.allclose(R.rotate64(x, at, freq, interleaved, 3.0)[..., :16], 3 * want[..., :16])
    # only the distance of two positions is in their product
    q, k = R.rotate64(x, at + 7, freq, interleaved), R.rotate64(x[::-1], at[::-1] + 7, freq, interleaved)
    q0, k0 = R.rotate64(x, at, freq, interleaved), R.rotate64(x[::-1], at[::-1], freq, interleaved)
    assert np.allclose((q * k).sum(-1), (q0 * k0).sum(-1))


def test_tree_sets_and_sees():
    parents = [-1, 0, 0, 1, 3, 2, 9, -1, 7]       # row 6 has no smaller parent: a root
    s = T.ancestors(parents)
    assert [list(np.flatnonzero(r)) for r in s] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5], [6],
                                                    [7], [7, 8]]
    w = T.words(s, 2)
    assert list(w[4]) == [0b11011, 0] and list(w[8]) == [0b110000000, 0]
    m = T.tree_sees(12, s)
    assert list(np.flatnonzero(m[5])) == [0, 1, 2, 3, 5, 8]
    assert list(np.flatnonzero(T.tree_sees(12, s, 4)[5])) == [2, 3, 5, 8]
    assert list(np.flatnonzero(T.tree_sees(12, s, 2)[5])) == [5, 8]
    assert not T.tree_sees(0, s).size
    assert list(np.flatnonzero(T.tree_sees(5, s)[4])) == [0]    # itself: rows 0 to 3 stand before the cache
    # a chain is the causal mask
    from oracle import msq_kv as O
    c = T.ancestors(np.arange(6) - 1)
    for window in (0, 1, 3, 8, 30):
        assert np.array_equal(T.tree_sees(20, c, window), O.sees(20, 6, True, window))


def test_verify_worked():
    p = np.array([[.5, .3, .2, 0], [.1, .1, .1, .7], [.25, .25, .25, .25]])
    u = np.array([.6, .2, .9], np.float32)
    # row 1 (token 0, u .2 < .5) is taken, row 2 below it (token 3, .9 > .7) is not: of the rest .1 each
    assert T.verify([9, 0, 3], None, p, None, u) == (1, [0, 1])
    # siblings: token 1 not taken (.9 > .3), token 0 of what is left: .2 * .7 < .5
    assert T.verify([9, 1, 0], [-1, 0, 0], p, None, np.array([.6, .9, .2], np.float32)) == (2, [0, 2])
    # the same token again has nothing left; then 0 and 2 by .5 and .2
    assert T.verify([9, 1, 1], [-1, 0, 0], p, None, np.array([.8, .9, 0], np.float32)) == (2, [0])
    # drawn from q: token 2 has .2 / .8; the rest is max(p - q, 0) = (.4, .2, 0, 0)
    q = np.array([[.1, .1, .8, 0]] * 3)
    assert T.verify([9, 2], None, p[:2], q[:2], np.array([.5, .3], np.float32)) == (0, [0])
    assert T.verify([9, 2], None, p[:2], q[:2], np.array([.7, .3], np.float32)) == (1, [0])
    assert T.verify([9, 2], None, p[:2], q[:2], np.array([.95, .2], np.float32)) == (3, [0, 1])
    # largest entries, ties to the first
    assert T.verify([9, 0, 3, 0], [-1, 0, 1, 2], np.vstack([p, p[2:]])) == (0, [0, 1, 2, 3])
    assert T.verify([], None, p[:0], None, u[:0]) == (-1, [])


def border(holds):
    """The length of the numbers in [0, 1] for which holds(u), true up to some number only; by halving."""
    lo, hi = 0.0, 1.0
    for _ in range(40):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if holds(mid) else (lo, mid)
    return lo


@pytest.mark.parametrize("draft", [True, False])
def test_verify_keeps_the_targets_probabilities(draft):
    """The first token after the certain one is the target's: summed over all drafts of two siblings and,
    for each, over the lengths of the intervals of the random numbers that lead to it (within 2^-39 each)."""
    p, q = np.array([.15, .35, .05, .45]), np.array([.4, .1, .3, .2])
    target, qs = np.stack([p] * 3), np.stack([q] * 3)
    got = np.zeros(4)
    drafts = [((x, y), q[x] * q[y]) for x in range(4) for y in range(4)] if draft else [((2, 1), 1.0)]
    for (x, y), weight in drafts:
        run = lambda v, u, w: T.verify([0, x, y], [-1, 0, 0], target, qs if draft else None, [v, u, w])
        one = border(lambda u: 1 in run(0.5, u, 0.5)[1])
        two = border(lambda w: 2 in run(0.5, 1.0, w)[1])
        got[x] += weight * one
        got[y] += weight * (1 - one) * two
        upto = [border(lambda v: run(v, 1.0, 1.0)[0] <= t) for t in range(4)]
        got += weight * (1 - one) * (1 - two) * np.diff([0.0] + upto)
    assert np.abs(got - p).max() < 1e-9
