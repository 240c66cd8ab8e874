"""Rotary positions on the GPU against their definition in 64 bits, forward and inverse, and as a gradient."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from _util import bits, ensure_built
from oracle import check, paged

pytestmark = pytest.mark.gpu

# A rotated value is off, before its one rounding to bf16, by: an angle of 2^-32 of a turn (1.5e-9) and the rounding of
# that angle to 24 bits (at most 2^-24 of pi, 1.9e-7); 2 units of 2^-24 in the sine and cosine (1.2e-7), half a unit for
# the factor (6e-8); and two roundings of half a unit in the products and their sum (1.2e-7).  Each acts on
# |x_a| + |x_b|: 4.9e-7 in all, 2^-20.9.
TOL = 2.0 ** -20


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def near(got_bits, ref, size):
    r = check.compare(got_bits, ref, TOL * size.ravel())
    assert r["ok"], r


def case(n, heads, d, dims, pos, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, heads, d), generator=gen, device="cuda").to(torch.bfloat16)
    inv = (10000.0 ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)).float().cuda()
    return x, torch.tensor(pos, dtype=torch.int32, device="cuda"), inv


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n, heads, d, dims", [(1, 1, 128, 128), (7, 5, 256, 256), (33, 40, 128, 64), (5, 17, 256, 48),
                                               (130, 3, 128, 16), (2, 64, 256, 240)])
def test_rotation(wa, n, heads, d, dims, layout, inverse):
    pos = np.random.default_rng(n).integers(0, 200000, n).tolist()
    x, p, inv = case(n, heads, d, dims, pos, seed=dims + n)
    out = wa.rope(x, p, inv, layout=layout, factor=1.25, inverse=inverse)
    ref, size = paged.rotate(oracle.bf16_to_f64(bits(x)), pos, inv.cpu().numpy(), layout, 1.25, inverse)
    near(bits(out), ref, size)
    assert torch.equal(out[..., dims:], x[..., dims:])


def test_far_and_negative_positions(wa):
    pos = [0, 1, -1, 10 ** 6 + 1, -123456789, 2 ** 31 - 1, -2 ** 31, 999999937]
    x, p, inv = case(len(pos), 2, 128, 128, pos, seed=5)
    ref, size = paged.rotate(oracle.bf16_to_f64(bits(x)), pos, inv.cpu().numpy(), "half")
    # the oracle's own angle, a float64 of up to 2^31, is off by 2^-22 of a radian at most
    r = check.compare(bits(wa.rope(x, p, inv)), ref, (TOL + 2.0 ** -22) * size.ravel())
    assert r["ok"], r


def test_odd_frequencies(wa):
    """Zero, subnormal, negative, above one, below 16; 16, infinities and NaN give NaN to their pairs alone."""
    w = [0.0, 1e-40, -0.75, 3.5, 15.999, 16.0, float("inf"), float("nan")]
    x, p, _ = case(6, 2, 128, 16, [0, 1, 5, 1000, 70001, 2 ** 24 + 1], seed=6)
    inv = torch.tensor(w, device="cuda")
    out = wa.rope(x, p, inv, layout="interleaved")
    ref, size = paged.rotate(oracle.bf16_to_f64(bits(x)), p.tolist(), inv.cpu().numpy()[:5], "interleaved")
    near(bits(out[..., :10]), ref[..., :10], size[..., :10])
    assert torch.isnan(out[..., 10:16]).all() and torch.equal(out[..., 16:], x[..., 16:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_in_the_projection_rows(wa, layout):
    """Queries and keys of interleaved rows turned in place: the same bits, the values untouched."""
    n, hq, hkv, d = 37, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randn((n, (hq + 2 * hkv) * d + 64), generator=gen, device="cuda").to(torch.bfloat16)
    _, p, inv = case(n, 1, d, 96, list(range(500, 500 + n)), seed=9)
    before = rows.clone()
    x = rows[:, :(hq + hkv) * d].view(n, hq + hkv, d)
    want = wa.rope(x, p, inv, layout=layout)
    assert wa.rope(x, p, inv, layout=layout, out=x) is x
    assert torch.equal(x, want) and torch.equal(rows[:, (hq + hkv) * d:], before[:, (hq + hkv) * d:])


def test_gradient_is_the_inverse(wa):
    """<g, R x> = <R^T g, x>, and R^T g against differences of the definition along single inputs."""
    n, heads, d, dims, f = 3, 2, 128, 64, 1.5
    x, p, inv = case(n, heads, d, dims, [4, 777, 70000], seed=10)
    g, _, _ = case(n, heads, d, dims, [0] * n, seed=11)
    dx = wa.rope(g, p, inv, factor=f, inverse=True)
    gf, xf, w, pos = oracle.bf16_to_f64(bits(g)), oracle.bf16_to_f64(bits(x)), inv.cpu().numpy(), p.tolist()
    ref, size = paged.rotate(gf, pos, w, "half", f, True)
    near(bits(dx), ref, size)
    rng = np.random.default_rng(12)
    for _ in range(20):
        i = tuple(rng.integers(0, m) for m in x.shape)
        h = np.zeros(x.shape)
        h[i] = 0.5
        up, down = (paged.rotate(xf + s * h, pos, w, "half", f)[0] for s in (1, -1))
        slope = ((up - down) * gf).sum()
        # dx is that slope rounded to bf16 (2^-9 of it) with the tolerance above
        assert abs(float(dx[i]) - slope) <= 2.0 ** -8 * abs(slope) + TOL * size[i] + 1e-9


def test_on_another_stream_and_in_a_graph(wa):
    x, p, inv = case(64, 48, 128, 128, list(range(64)), seed=13)
    want = wa.rope(x, p, inv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = wa.rope(x, p, inv, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, g = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wa.rope(x, p, inv, out=out)
    p.add_(100)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, wa.rope(x, p, inv))
