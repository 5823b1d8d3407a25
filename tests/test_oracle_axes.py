"""The rotation by positions on several axes (oracle/heads.py): pinned by what defines it."""
import numpy as np
import pytest

from oracle import heads as H

AXIS = [0, 0, 1, 2, 1, 2, 0, 1]
FREQ = 100.0 ** (-np.arange(8) / 8)


def test_equal_positions_on_all_axes_are_one_position():
    p = np.array([0, 3, 17, 40000])
    np.testing.assert_array_equal(H.axis_phases(np.stack([p] * 3, -1), AXIS, FREQ), H.phases(p, FREQ))


def test_a_pair_turns_by_its_axis_alone():
    pos = np.array([[5, 7, 11]])
    z = H.axis_phases(pos, AXIS, FREQ)
    for i, a in enumerate(AXIS):
        assert z[0, i] == pytest.approx(np.exp(1j * pos[0, a] * FREQ[i]), abs=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_scores_depend_on_the_differences_of_positions(inter):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 6, 1, 20))  # four elements are not rotated
    pq, pk, by = rng.integers(0, 50, (6, 3)), rng.integers(0, 50, (6, 3)), np.array([9, -4, 30])

    def score(p1, p2):
        a, b = H.turn(q, H.axis_phases(p1, AXIS, FREQ), inter), H.turn(k, H.axis_phases(p2, AXIS, FREQ), inter)
        return (a * b).sum(-1)
    np.testing.assert_allclose(score(pq + by, pk + by), score(pq, pk), atol=1e-12)
    assert np.abs(score(pq + by, pk) - score(pq, pk)).max() > 0.1


def test_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((5, 2, 16)), rng.standard_normal((5, 2, 16)), rng.standard_normal(16)
    z = H.axis_phases(rng.integers(-20, 20, (5, 3)), AXIS, FREQ)
    dx, dw = H.norm_rope_bwd(dy, x, w, z, 1e-3)
    loss = lambda x, w: (H.norm_rope_fwd(x, w, z, 1e-3) * dy).sum()  # noqa: E731
    h = 1e-6
    for at in [(0, 0, 0), (3, 1, 15), (4, 0, 7)]:
        e = np.zeros_like(x)
        e[at] = h
        assert dx[at] == pytest.approx((loss(x + e, w) - loss(x - e, w)) / (2 * h), abs=1e-7)
    for i in (0, 9):
        e = np.zeros_like(w)
        e[i] = h
        assert dw[i] == pytest.approx((loss(x, w + e) - loss(x, w - e)) / (2 * h), abs=1e-7)
