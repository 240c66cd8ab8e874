"""Serving steps over a paged cache, the operators together: a prompt's chunk appended, then tokens one by one, each
step's attention against the ring cache's decode over the same keys and values."""
from __future__ import annotations

import pytest
import torch

import oracle
from _util import bits, ensure_built
from oracle import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("win", [0, 96])
def test_steps_agree_with_the_ring_cache(wa, win):
    rows, hq, hkv, d, page, most = 3, 8, 2, 128, 16, 20
    start, steps = [130, 1, 47], 4
    gen = torch.Generator(device="cuda").manual_seed(60)
    inv, factor = wa.rope_frequencies(d, scaling={"kind": "linear", "factor": 2}, device="cuda")
    table = torch.randperm(rows * most, generator=torch.Generator().manual_seed(61)).int().view(rows, most).cuda()
    k, v = (torch.zeros((rows * most, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k_ring, v_ring = (torch.zeros((rows, page * most, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    width = (hq + 2 * hkv) * d

    def put(x, pos, row, q):
        """Into the pages by the append; into the rings by the rotation alone."""
        ws = wa.paged_append(x, pos, q, k, v, table, row=row, inv_freq=inv, factor=factor)
        assert wa.status(ws) == 0
        heads = x.view(len(x), hq + 2 * hkv, d)
        turned = wa.rope(heads[:, :hq + hkv], pos, inv, factor=factor)
        assert torch.equal(turned[:, :hq], q)
        k_ring[row.long(), pos.long()] = turned[:, hq:]
        v_ring[row.long(), pos.long()] = heads[:, hq + hkv:]

    # the prompts' chunks together
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in start]).cuda()
    row = torch.cat([torch.full((n,), r, dtype=torch.int32) for r, n in enumerate(start)]).cuda()
    x = torch.randn((len(pos), width), generator=gen, device="cuda").to(torch.bfloat16)
    put(x, pos, row, torch.empty((len(pos), hq, d), dtype=torch.bfloat16, device="cuda"))
    at = torch.tensor(start, dtype=torch.int32, device="cuda")
    every = torch.arange(rows, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        x = torch.randn((rows, width), generator=gen, device="cuda").to(torch.bfloat16)
        q = torch.empty((rows, hq, d), dtype=torch.bfloat16, device="cuda")
        put(x, at, every, q)
        got = wa.paged_decode(q, k, v, table, at, win=win, scale=d ** -0.5)
        ref = oracle.decode(bits(q), bits(k_ring), bits(v_ring), at.tolist(), win, page * most, d ** -0.5)
        r = check.compare(bits(got), ref, check.TOL_FP32_P)
        assert r["ok"], r
        ring = wa.decode(q, k_ring, v_ring, at, win, d ** -0.5)
        r = check.compare(bits(ring), ref, check.TOL_FP32_P)
        assert r["ok"], r
        at += 1
