"""What the drafted-token calls allocate, where the caller names a stream that is not the current one."""
from __future__ import annotations

import pytest
import torch

import wa_synth
from _util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def _calls(wa):
    """name -> (call(stream) -> its new tensors, their sizes in bytes)"""
    c = wa_synth.tree_case(9, 30, 16, 4, 256, 0, 900, [899 - 90 * r for r in range(9)], seed=51, device="cuda",
                           outside="keep")
    gen = torch.Generator(device="cuda").manual_seed(52)
    target = torch.softmax(torch.randn((9, 30, 2000), generator=gen, device="cuda"), -1)
    tokens = torch.randint(0, 2000, (9, 30), generator=gen, device="cuda").int()
    u = torch.rand((9, 30), generator=gen, device="cuda")
    zeros = torch.zeros((9, 30), dtype=torch.int32, device="cuda")
    return {
        "decode": lambda s: [wa.tree_decode(c["q"], c["k"], c["v"], c["k_tree"], c["v_tree"], c["pos"], c["parent"], 0,
                                            scale=0.06, stream=s)],
        "verify": lambda s: list(wa.tree_verify(target, c["parent"], tokens, u, stream=s)),
        "commit": lambda s: [wa.tree_commit(c["k_tree"], c["v_tree"], c["k"].clone(), c["v"].clone(), zeros,
                                            zeros[:, 0].contiguous(), c["pos"], stream=s)],
    }


@pytest.mark.parametrize("name", ["decode", "verify", "commit"])
def test_allocations_come_from_the_streams_own_memory(wa, name):
    """Memory that was freed on the current stream may still be written by what is queued there: a call on another
    stream, which does not wait for it, must not be given that memory."""
    call, s = _calls(wa)[name], torch.cuda.Stream()
    sizes = [t.untyped_storage().nbytes() for t in call(None)]
    torch.cuda.synchronize()
    held = [[torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)] for n in sizes]
    freed = {t.data_ptr() for ts in held for t in ts}
    del held
    got = call(s)
    torch.cuda.synchronize()
    assert not freed & {t.data_ptr() for t in got}


@pytest.mark.parametrize("name", ["decode", "verify"])
def test_results_beside_work_that_is_still_queued(wa, name):
    """The current stream sleeps, then writes memory that is free by then; a call on another stream meanwhile."""
    call, s = _calls(wa)[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)        # about 0.1 s
    junk = [torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device="cuda") for t in want for _ in range(4)]
    for x in junk:
        x.fill_(0xAB)
    del junk
    x = None
    got = call(s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_captured_calls_that_allocate(wa):
    """A call without an output or a workspace inside a capture, by either way in."""
    calls, s = _calls(wa), torch.cuda.Stream()
    want = {n: calls[n](None) for n in ("decode", "verify")}
    torch.cuda.synchronize()
    for stream in (None, s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = {n: calls[n](stream) for n in want}
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got[n], want[n])), n


def test_without_the_extension_module(wa, monkeypatch):
    """The same bits by way of ctypes alone."""
    calls = _calls(wa)
    want = {n: calls[n](None) for n in ("decode", "verify")}
    monkeypatch.setattr(wa, "_bind", None)
    for n, ts in want.items():
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(calls[n](None), ts)), n
