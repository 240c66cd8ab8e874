"""What a part of P less would do to the outputs that the paged decode's precision tests look at (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from _paged_precision import cancelling, weights


@pytest.mark.parametrize("bits, parts, bound", [(16, 2, 2.0 ** -17), (8, 3, 2.0 ** -14)])
def test_a_part_less_is_seen(bits, parts, bound):
    """The bounds that the library states for P hold with all its parts, and one part less is past twice them in many dims."""
    for seed in range(6):
        t, v = cancelling(256, seed)
        w = np.exp(t)
        size, exact = (w @ np.abs(v)) / w.sum(), (w @ v) / w.sum()
        assert (np.abs(exact) < 2.0 ** -11).all()
        off = [np.abs((weights(t, n, bits) @ v) / w.sum() - exact) for n in (parts, parts - 1)]
        assert (off[0] <= bound * size).all()
        assert (off[1] > 2 * bound * size).mean() > 0.1


@pytest.mark.parametrize("bits, parts, bound, least", [(16, 2, 2.0 ** -17, 0.0), (8, 3, 2.0 ** -14, 2.0 ** -28)])
def test_a_weights_error(bits, parts, bound, least):
    """Weights down to 2^-40 of the largest: within the stated part of the weight, or of the largest."""
    t = -np.random.default_rng(7).uniform(0, 27, 200000)
    off = np.abs(weights(t, parts, bits) - np.exp(t))
    assert (off <= np.maximum(bound * np.exp(t), least)).all()
