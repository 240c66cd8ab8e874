"""What the paged decode keeps of its probabilities, queries and scores, on the GPU, at inputs that show it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import wa_synth
from _paged_precision import LIVE, cancelling, place
from _util import bits, ensure_built
from oracle import check
from test_paged_decode_gpu import call, reference, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("hq, hkv", [(4, 2), (8, 1), (13, 1)])      # groups of up to 4, 8 and 16 heads
@pytest.mark.parametrize("bits_, d", [(16, 128), (16, 256), (8, 128), (8, 256)])
@pytest.mark.parametrize("e", [13, 15, 17, 18, 19, 20, 22, 25])
def test_scores_of_any_size(wa, e, bits_, d, hq, hkv):
    """Scores of 2^(e + 8) to 2^(e + 9), in units of log2, whose fp32 neighbours are up to 2^10 apart.  A key that is alone, or whose
    score is that far above all others, has weight 1, and the output is its value: nothing is rounded."""
    lengths = [1, 200, 3] * 12
    c = wa_synth.paged_case(lengths, hq, hkv, d, 16, seed=80, bits=bits_, device="cuda", outside="keep", peaked=False)
    c["k_scale"] = c["v_scale"] = None
    c["q"].zero_()
    c["k"].copy_(torch.zeros((), device="cuda"))
    for r, n in enumerate(lengths):              # the last key of a sequence
        c["k"][int(c["table"][r, (n - 1) // 16]), (n - 1) % 16, :, 0] = torch.ones((), device="cuda").to(c["k"].dtype)
    m = torch.arange(len(lengths) * hq, device="cuda") * 37 % 128        # all 8-bit significands
    c["q"][:, :, 0] = ((128 + m) * 2.0 ** e).view(len(lengths), hq).to(torch.bfloat16)
    r = check.compare(bits(call(wa, c, 2.0 ** 0.5)), reference(c, 2.0 ** 0.5), 0.0)
    assert r["ok"], r
    one = [i for i, n in enumerate(lengths) if n == 1]      # and that far below zero
    c = dict(c, q=c["q"][one], table=c["table"][one], pos=c["pos"][one])
    r = check.compare(bits(call(wa, c, -(2.0 ** 0.5))), reference(c, -(2.0 ** 0.5)), 0.0)
    assert r["ok"], r


def near(got, exact, off):
    """Outputs within `off` of 64-bit values before their rounding to bf16 (half a step: 2^-8 of the value)."""
    got = oracle.bf16_to_f64(bits(got))
    over = np.abs(got - exact) - (off + 2.0 ** -8 * (np.abs(exact) + off))
    assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("hq, hkv", [(4, 1), (16, 2), (16, 1), (12, 1)])
@pytest.mark.parametrize("bits_, bound", [(16, 2.0 ** -17), (8, 2.0 ** -14)])
@pytest.mark.parametrize("d", [128, 256])
def test_probabilities_keep_their_parts(wa, d, bits_, bound, hq, hkv):
    """Values that cancel: what the weights lose is the output's error, of size sum_j w_j |v_j| / sum_j w_j.

    Besides the bound for P, 2^-19 of that size: a score in units of log2 of up to 1.45 is off by 2^-23 of it (its factor's
    rounding and its own), with 8 added to it by 2^-22, in a weight both times ln 2, 2^-22.1; the exponential 2^-22; and the
    eight products' sum by 2^-24 or, where a tensor core cuts off, 2^-23 a step, 2^-20."""
    seeds, rng = range(4), np.random.default_rng(d + hq)
    lengths = [128, 1000, 700, 129]
    c = wa_synth.paged_case(lengths, hq, hkv, d, 16, seed=81, bits=bits_, device="cuda", outside="keep", peaked=False)
    sets = [cancelling(d, s) for s in seeds]
    first = [0, 512, 384, 0]
    place(c, [f + rng.choice(128, LIVE, replace=False) for f in first], [t for t, _ in sets], [v for _, v in sets])
    out = call(wa, c).cpu()
    for r, (t, v) in enumerate(sets):
        w = np.exp(t)
        near(out[r], np.broadcast_to(w @ v / w.sum(), (hq, d)), (bound + 2.0 ** -19) * (w @ np.abs(v) / w.sum()))


@pytest.mark.parametrize("hq, hkv", [(4, 1), (16, 2), (16, 1), (9, 1)])
@pytest.mark.parametrize("d", [128, 256])
def test_a_query_with_one_large_value(wa, d, hq, hkv):
    """Over 8-bit pages a query's value is a sum of 8-bit numbers, within 2^-21 of its head's largest value.  The largest stands
    where every key is zero, the scores come from one value of about 2^-12 of it.  With every score off by at most x, weights
    are off by a factor of e^(2 x) of one another at most."""
    c = wa_synth.paged_case([40, 300, 1, 1100], hq, hkv, d, 32, seed=82, bits=8, device="cuda", outside="keep", peaked=False)
    gen = torch.Generator(device="cuda").manual_seed(83)
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    c["q"][:, :, 1] = ((1 + torch.rand((4, hq), generator=gen, device="cuda")) * 2.0 ** -12).to(torch.bfloat16)
    k = torch.zeros(c["k"].shape, device="cuda")
    k[..., 1] = torch.randint(-8, 9, k.shape[:-1], generator=gen, device="cuda").float()
    c["k"].copy_(k)
    c["k_scale"], c["v_scale"] = torch.full((hkv,), 1024.0, device="cuda"), None
    ref = reference(c, 1.0)
    off = np.exp(2 * 8 * 1024 * 2.0 ** -21) - 1
    # sum_j w_j |v_j| / sum_j w_j; scores of up to 8 (11.6 in units of log2: 2^-19.3 in a weight) and weights within 2^-14
    size = reference(dict(c, v=torch.from_numpy(np.abs(stored(c["v"]))).cuda().float().to(c["v"].dtype)), 1.0)
    near(call(wa, c), ref, (off + 2.0 ** -14 + 2.0 ** -18) * size)
