"""Frequencies that the rotation does not take are refused where they are made (CPU)."""
from __future__ import annotations

import math

import pytest

import sliding_window_gqa_gb300 as wa


@pytest.mark.parametrize("scaling", [
    {"kind": "linear", "factor": 0.05}, {"kind": "linear", "factor": 1 / 16}, {"kind": "wavelength", "factor": 0.01, "original": 4},
    {"kind": "ramp", "factor": 0.01, "original": 8, "fast": 1000.0}, {"kind": "base", "factor": 1e-9},
], ids=str)
def test_a_fastest_pair_of_16_and_more_is_refused(scaling):
    """(The rotation gives NaN for pairs of frequency 16 and above.)"""
    with pytest.raises(ValueError, match="16"):
        wa.rope_frequencies(64, scaling=scaling)


def test_what_is_just_below_is_not():
    inv, _ = wa.rope_frequencies(64, scaling={"kind": "linear", "factor": 1 / 15.99})
    assert math.isclose(float(inv[0]), 15.99, rel_tol=1e-6)
    inv, _ = wa.rope_frequencies(64, scaling={"kind": "linear", "factor": 1 / math.nextafter(16.0, 0.0) * (1 + 2.0 ** -20)})
    assert float(inv[0]) < 16.0
