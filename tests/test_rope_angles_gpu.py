"""How exact the rotation's angles are, seen where a sine or cosine is next to zero."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from _util import bits, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_next_to_quarters_of_a_turn(wa, layout):
    """Frequency 1 at the positions nearest to whole quarters of a turn: there a sine or cosine of 3e-7 to 1e-3 is the angle's own
    distance from the quarter, and bf16 keeps it to half a step (2^-8 of it).

    An angle is a fraction of a turn cut to 32 bits (2^-32, and 2^-33 before that), then rounded to fp32, by 2^-26 at
    most, next to half a turn: 2^-25.9 of a turn together.  The sine and cosine are within 2^-22 of themselves."""
    k = np.arange(1, 4_000_000, dtype=np.float64)
    pos = np.concatenate([np.argsort(np.abs(f(k)))[:200] + 1 for f in (np.cos, np.sin)]).astype(np.int64)
    pos = np.concatenate([pos, -pos])
    x = torch.zeros((len(pos), 1, 128), dtype=torch.bfloat16, device="cuda")
    x[..., 0] = 1.0
    inv = torch.zeros(64, device="cuda")
    inv[0] = 1.0
    y = oracle.bf16_to_f64(bits(wa.rope(x, torch.from_numpy(pos).int().cuda(), inv, layout=layout)))[:, 0]
    other = 64 if layout == "half" else 1
    for got, ref in ((y[:, 0], np.cos(pos.astype(np.float64))), (y[:, other], np.sin(pos.astype(np.float64)))):
        off = 2 * np.pi * 2.0 ** -25.9 + 2.0 ** -22 * np.abs(ref)
        over = np.abs(got - ref) - (off + 2.0 ** -8 * (np.abs(ref) + off))
        assert (over <= 0).all(), (over.max(), pos[over.argmax()])
    assert not y[:, [i for i in range(128) if i not in (0, other)]].any()
