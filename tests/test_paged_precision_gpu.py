"""What the paged decode keeps of its probabilities, queries and scores, on the GPU, at inputs that show it."""
from __future__ import annotations

import pytest
import torch

import wa_synth
from _util import bits, ensure_built
from oracle import check
from test_paged_decode_gpu import call, reference

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
