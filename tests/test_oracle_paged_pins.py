"""Pins of the paged-cache oracle (CPU): the 8-bit type against torch's, the rotation against complex numbers, the
decode against one contiguous cache; and the frequencies that the package works out for long contexts."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import sliding_window_gqa_gb300 as wa
import wa_synth
from _util import bits
from oracle import paged


def test_e4m3_values_and_rounding_against_torch():
    every = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(paged.e4m3_to_f64(every), want)
    x = np.concatenate([np.random.default_rng(1).normal(0, s, 4000) for s in (1e-3, 0.1, 3.0, 200.0)])
    fine = want[np.isfinite(want)]
    x = np.concatenate([x, fine, (np.sort(fine)[1:] + np.sort(fine)[:-1]) / 2, [1e9, -1e9, np.inf, 448, 464, 465]])
    x = x.astype(np.float32).astype(np.float64)
    got = paged.f64_to_e4m3(x)
    ref = torch.from_numpy(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    same = (got == ref) | ((got & 0x7F == 0) & (ref & 0x7F == 0))
    assert same.all(), x[~same][:5]
    assert paged.f64_to_e4m3(np.array([np.nan]))[0] & 0x7F == 0x7F


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_multiplication_by_a_unit_complex_number(layout):
    rng = np.random.default_rng(2)
    x, pos, inv = rng.normal(size=(5, 3, 32)), np.array([0, 1, -7, 90001, 2 ** 30]), 10.0 ** -np.arange(8)
    y, _ = paged.rotate(x, pos, inv, layout, factor=1.5)
    a, b = (slice(0, 8), slice(8, 16)) if layout == "half" else (slice(0, 16, 2), slice(1, 16, 2))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None] * inv)[:, None] * 1.5
    np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
    back, _ = paged.rotate(y, pos, inv, layout, factor=1 / 1.5, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_decode_over_pages_is_decode_over_a_line():
    c = wa_synth.paged_case([70, 1, 0, 33], 6, 2, 128, 16, seed=3, win=40)
    k, v = (oracle.bf16_to_f64(bits(c[x])) for x in "kv")
    got = paged.decode(oracle.bf16_to_f64(bits(c["q"])), k, v, c["table"].numpy(), c["pos"].numpy(), 40, 0.7)
    for r, n in enumerate([70, 1, 0, 33]):
        if n == 0:
            assert not got[r].any()
            continue
        line = [np.zeros((1, n, 2, 128), dtype=np.uint16) for _ in "kv"]
        for at in range(max(0, n - 40), n):
            for x, src in zip(line, (bits(c["k"]), bits(c["v"]))):
                x[0, at] = src[int(c["table"][r, at // 16]), at % 16]
        want = oracle.decode(bits(c["q"])[r:r + 1], *line, [n - 1], 40, n, 0.7) if n > 40 else \
            oracle.decode(bits(c["q"])[r:r + 1], *line, [n - 1], 0, n, 0.7)
        np.testing.assert_allclose(got[r], want[0], atol=1e-12)
    assert np.isfinite(got).all()


def test_append_leaves_out_what_has_no_place():
    table = np.array([[2, -1], [0, 1]])
    x = np.arange(4 * 3 * 16, dtype=np.float64).reshape(4, 3, 16)
    _, _, places = paged.append(x, [5, 17, -1, 31], [0, 0, 1, 1], 1, 1, table, 16, k_scale=[2.0])
    assert [(p, s) for p, s, *_ in places] == [(2, 5), (1, 15)]
    np.testing.assert_array_equal(places[1][2][0], x[3, 1] / 2)
    np.testing.assert_array_equal(places[1][4][0], x[3, 2])


def test_frequencies_for_long_contexts():
    plain, one = wa.rope_frequencies(128, 500000.0)
    assert one == 1.0 and plain.dtype == torch.float32 and plain.shape == (64,)
    np.testing.assert_array_equal(plain.numpy(), (500000.0 ** (-np.arange(0, 128, 2) / 128)).astype(np.float32))
    linear, _ = wa.rope_frequencies(128, 500000.0, {"kind": "linear", "factor": 4})
    np.testing.assert_array_equal(linear.numpy(), (500000.0 ** (-np.arange(0, 128, 2) / 128) / 4).astype(np.float32))
    stretched, _ = wa.rope_frequencies(128, 500000.0, {"kind": "base", "factor": 4})
    assert stretched[0] == 1.0 and math.isclose(stretched[-1], plain[-1] / 4, rel_tol=1e-6)
    # turns over the original length: above `high` as they are, below `low` divided, in between between
    w, _ = wa.rope_frequencies(128, 500000.0, {"kind": "wavelength", "factor": 8, "original": 8192})
    turns = 8192 * plain.double() / (2 * math.pi)
    assert torch.equal(w[turns > 4], plain[turns > 4])
    assert torch.allclose(w[turns < 1], plain[turns < 1] / 8, rtol=1e-6)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((w[mid] < plain[mid]) & (w[mid] > plain[mid] / 8)).all()
    r, grow = wa.rope_frequencies(64, 10000.0, {"kind": "ramp", "factor": 16, "original": 4096})
    turns = 4096 * (10000.0 ** (-np.arange(0, 64, 2) / 64)) / (2 * math.pi)
    plain = wa.rope_frequencies(64)[0].numpy()
    assert math.isclose(grow, 0.1 * math.log(16) + 1)
    np.testing.assert_array_equal(r.numpy()[turns > 40], plain[turns > 40])
    np.testing.assert_allclose(r.numpy()[turns < 0.7], plain[turns < 0.7] / 16, rtol=1e-6)
    assert (np.diff(r.numpy()) < 0).all()
    assert wa.rope_frequencies(64, scaling={"kind": "ramp", "factor": 16, "original": 4096, "attention": 1.25})[1] == 1.25


@pytest.mark.parametrize("bad", [
    dict(dims=0), dict(dims=7), dict(dims=64, base=0.5), dict(dims=64, base=float("inf")),
    dict(dims=64, scaling={"kind": "cubic", "factor": 2}), dict(dims=64, scaling={"kind": "linear"}),
    dict(dims=64, scaling={"kind": "linear", "factor": 0}), dict(dims=64, scaling={"kind": "linear", "factor": 2, "base": 3}),
    dict(dims=2, scaling={"kind": "base", "factor": 2}), dict(dims=64, scaling={"kind": "ramp", "factor": 2}),
    dict(dims=64, scaling={"kind": "wavelength", "factor": 2, "original": 4096, "low": 4, "high": 4}),
    dict(dims=64, scaling={"factor": 2}),
], ids=str)
def test_frequencies_that_are_refused(bad):
    with pytest.raises(ValueError):
        wa.rope_frequencies(**bad)


def test_scaling_of_another_type_is_refused():
    with pytest.raises(TypeError):
        wa.rope_frequencies(64, scaling="linear")
