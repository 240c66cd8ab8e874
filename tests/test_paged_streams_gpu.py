"""The rotary and paged-cache calls on streams: their own allocations, kernels launched while the one before runs, captured
steps, and the same bits by either way in."""
from __future__ import annotations

import pytest
import torch

import oracle
import wa_synth
from _util import bits, ensure_built
from oracle import check, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def _calls(wa):
    """name -> (call(stream) -> its new tensors)"""
    c = wa_synth.paged_case([900, 3, 0, 4000], 16, 4, 256, 32, seed=70, device="cuda", outside="keep", bits=8)
    gen = torch.Generator(device="cuda").manual_seed(71)
    src = torch.randn((4, 24 * 256), generator=gen, device="cuda").to(torch.bfloat16)
    inv, _ = wa.rope_frequencies(256, device="cuda")
    pos = torch.tensor([899, 2, -1, 3999], dtype=torch.int32, device="cuda")
    q = torch.empty((4, 16, 256), dtype=torch.bfloat16, device="cuda")

    def append(s):
        k, v = c["k"].clone(), c["v"].clone()
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        ws = wa.paged_append(src, pos, q, k, v, c["table"], inv_freq=inv, k_scale=c["k_scale"], v_scale=c["v_scale"], stream=s)
        return [ws, k, v]
    return {
        "rope": lambda s: [wa.rope(src[:, :20 * 256].unflatten(1, (20, 256)), pos, inv, stream=s)],
        "decode": lambda s: [wa.paged_decode(c["q"], c["k"], c["v"], c["table"], c["pos"], k_scale=c["k_scale"],
                                             v_scale=c["v_scale"], stream=s)],
        "append": append,
    }


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", ["rope", "decode", "append"])
def test_allocations_come_from_the_streams_own_memory(wa, name):
    """Memory freed on the current stream may still be written by what is queued there: not for a call on another one."""
    call, s = _calls(wa)[name], torch.cuda.Stream()
    size = call(None)[0].untyped_storage().nbytes()
    torch.cuda.synchronize()
    held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    freed = {t.data_ptr() for t in held}
    del held
    got = call(s)[0]
    torch.cuda.synchronize()
    assert got.data_ptr() not in freed


def test_without_the_extension_module(wa, monkeypatch):
    """The same bits by way of ctypes alone."""
    calls = _calls(wa)
    want = {n: f(None) for n, f in calls.items()}
    monkeypatch.setattr(wa, "_bind", None)
    for n, f in calls.items():
        got = f(None)
        assert wa.status(got[0]) == 0 if n == "append" else _same(got[0], want[n][0]), n
        assert all(_same(a, b) for a, b in zip(got[1:], want[n][1:])), n


def test_captured_calls_that_allocate(wa):
    calls, s = _calls(wa), torch.cuda.Stream()
    names = ("rope", "decode")
    want = {n: calls[n](None)[0] for n in names}
    torch.cuda.synchronize()
    for stream in (None, s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = {n: calls[n](stream)[0] for n in names}
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert all(_same(got[n], want[n]) for n in names)


@pytest.mark.parametrize("n", [3, 1500])
def test_layers_one_after_another(wa, n):
    """Each kernel starts while the one before it runs.  Layers of append, paged decode, rotation and the ring cache's
    decode, each reading what the call before has just written, in a row and captured, against the same calls with the GPU
    idle between them.  (n: tokens of an append, those of the status block and of the status kernel.)"""
    rows, hq, hkv, d, page, most, layers = 3, 8, 2, 128, 16, 40, 5
    gen = torch.Generator(device="cuda").manual_seed(72)
    inv, _ = wa.rope_frequencies(d, device="cuda")
    table = torch.randperm(rows * most, generator=torch.Generator().manual_seed(73)).int().view(rows, most).cuda()
    k, v = (torch.zeros((layers, rows * most, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    start = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    per = n // rows
    pos = torch.arange(per, dtype=torch.int32).repeat(rows).cuda()
    row = torch.arange(rows, dtype=torch.int32).repeat_interleave(per).cuda()
    last = torch.full((rows,), per - 1, dtype=torch.int32, device="cuda")
    x, q = torch.empty_like(start), torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    outs = torch.empty((layers, 3, rows, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    dws = torch.empty(wa.paged_decode_ws_bytes(rows, hq, hkv, d, page, most), dtype=torch.uint8, device="cuda")
    ring = torch.randn((2, rows, 512, hkv, d), generator=gen, device="cuda").to(torch.bfloat16)

    def run(between):
        x.copy_(start)
        for i in range(layers):
            wa.paged_append(x, pos, q, k[i], v[i], table, row=row, inv_freq=inv, ws=ws)
            between()
            tail = q[:rows]
            wa.paged_decode(tail, k[i], v[i], table, last, scale=d ** -0.5, out=outs[i, 0], ws=dws)
            between()
            wa.rope(outs[i, 0], last, inv, out=outs[i, 1])
            between()
            wa.decode(outs[i, 1], ring[0], ring[1], last, 0, d ** -0.5, out=outs[i, 2])
            between()
            heads = x[:, :hq * d].unflatten(1, (hq, d))
            wa.rope(heads, pos, inv, out=heads)
            between()

    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [t.clone() for t in (k, v, outs, x)]
    assert torch.isfinite(outs.float()).all() and outs.float().abs().sum() > 0

    def check_all():
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip((k, v, outs, x), want)) and wa.status(ws) == 0
        for t in (k, v, outs):
            t.zero_()

    for _ in range(10):
        run(lambda: None)
        check_all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for _ in range(10):
        g.replay()
        check_all()


def test_a_lone_head_in_a_pool_of_odd_page_strides(wa):
    """Pages of one key head, apart by a number of positions that 8 does not divide."""
    page, d, gap = 16, 128, 3
    c = wa_synth.paged_case([70, 1, 500], 4, 1, d, page, seed=74, device="cuda", outside="nan")
    sides = []
    for t in (c["k"], c["v"]):
        pool = torch.full((len(t) * (page + gap), d), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = pool.as_strided((len(t), page, 1, d), ((page + gap) * d, d, d, 1))
        view.copy_(t)
        sides.append(view)
    got = wa.paged_decode(c["q"], *sides, c["table"], c["pos"], scale=0.1)
    values = [oracle.bf16_to_f64(bits(t)) for t in sides]
    ref = paged.decode(oracle.bf16_to_f64(bits(c["q"])), *values, c["table"].cpu().numpy(), c["pos"].cpu().numpy(), 0, 0.1, None, None)
    r = check.compare(bits(got), ref, check.TOL_FP32_P)
    assert r["ok"], r
    assert _same(got, wa.paged_decode(c["q"], c["k"], c["v"], c["table"], c["pos"], scale=0.1))
