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


def test_a_token_changed_between_two_appends(wa):
    """The second of two large appends reads a few tokens that a small kernel between them has just written, and the rest
    again, with nothing else in between that would make an SM forget what it read for the first."""
    n, rows, hq, hkv, d, page = 1600, 4, 8, 2, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(75)
    inv, _ = wa.rope_frequencies(d, device="cuda")
    most = n // rows // page
    table = torch.arange(rows * most, dtype=torch.int32, device="cuda").view(rows, most)
    k, v = (torch.zeros((rows * most, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    start = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    x = start.clone()
    pos = torch.arange(n // rows, dtype=torch.int32).repeat(rows).cuda()
    row = torch.arange(rows, dtype=torch.int32).repeat_interleave(n // rows).cuda()
    one, two = (torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    few = x[777:781, :hq * d].unflatten(1, (hq, d))

    def run(between):
        wa.paged_append(x, pos, one, k, v, table, row=row, inv_freq=inv, ws=ws)
        between()
        wa.rope(few, pos[777:781], inv, out=few)
        between()
        wa.paged_append(x, pos, two, k, v, table, row=row, inv_freq=inv, ws=ws)

    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = one.clone(), two.clone()
    changed = (want[0] != want[1]).flatten(1).any(1)
    assert changed[777:781].all() and changed.sum() == 4
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            run(lambda: None)
    for way in (g.replay, lambda: [run(lambda: None) for _ in range(3)]):
        for _ in range(20):
            x.copy_(start)
            one.zero_(), two.zero_()
            run(lambda: None)
            torch.cuda.synchronize()
            assert _same(one, want[0]) and _same(two, want[1])
            # (each run turns the few tokens once more: the last append's queries are once more than the first's)
            before = few.clone()
            way()
            torch.cuda.synchronize()
            for _ in range(3):
                before = wa.rope(before, pos[777:781], inv)
            assert _same(few, before) and _same(two[777:781], wa.rope(before, pos[777:781], inv))


def test_a_capture_whose_branches_meet_at_a_call(wa):
    """Two branches of a captured graph, joined before a decode: it waits for both."""
    c = wa_synth.paged_case([400, 77], 8, 2, 128, 16, seed=76, device="cuda", outside="keep")
    want = [wa.paged_decode(q, c["k"], c["v"], c["table"], c["pos"], scale=0.1) for q in (c["q"], c["q"].flip(1))]
    q, k = torch.zeros_like(c["q"]), torch.zeros_like(c["k"])
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    src = [c["q"].clone(), c["k"].clone()]
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)            # about 0.1 ms
            k.copy_(src[1])
        q.copy_(src[0])
        main.wait_stream(side)
        out = wa.paged_decode(q, k, c["v"], c["table"], c["pos"], scale=0.1)
        k.zero_()
    for i in range(6):
        src[0].copy_(c["q"] if i % 2 == 0 else c["q"].flip(1))
        g.replay()
        torch.cuda.synchronize()
        assert _same(out, want[i % 2])


def test_layouts_of_the_pool_and_the_table(wa):
    """Keys and values side by side in the innermost dims, one heads first and the other not, and a table that is part of a
    wider one: the same bits as over plain pools."""
    for bits_ in (16, 8):
        c = wa_synth.paged_case([300, 1, 0, 1111], 12, 3, 128, 32, seed=77, device="cuda", bits=bits_, outside="nan")
        call = lambda k, v, table: wa.paged_decode(c["q"], k, v, table, c["pos"], scale=0.1, k_scale=c["k_scale"], v_scale=c["v_scale"])
        want = call(c["k"], c["v"], c["table"])
        pages, page, hkv, d = c["k"].shape
        inner = torch.empty((pages, page, hkv, 2, d), dtype=c["k"].dtype, device="cuda")
        inner[:, :, :, 0], inner[:, :, :, 1] = c["k"], c["v"]
        first = c["k"].transpose(1, 2).contiguous().transpose(1, 2)
        wide = torch.full((4, c["table"].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
        wide[:, 2:-3] = c["table"]
        assert _same(call(inner[:, :, :, 0], inner[:, :, :, 1], c["table"]), want)
        assert _same(call(first, c["v"], c["table"]), want)
        assert _same(call(c["k"], first.copy_(c["v"]), wide[:, 2:-3]), want)


@pytest.mark.parametrize("hq, hkv", [(64, 64), (40, 20), (16, 1)])
def test_many_key_heads_and_few(wa, hq, hkv):
    """As many key heads as query heads, groups of two, and one for all."""
    for bits_ in (16, 8):
        c = wa_synth.paged_case([1, 260, 900], hq, hkv, 128, 64, seed=78, device="cuda", bits=bits_)
        got = wa.paged_decode(c["q"], c["k"], c["v"], c["table"], c["pos"], scale=0.1, k_scale=c["k_scale"], v_scale=c["v_scale"])
        values = [oracle.bf16_to_f64(bits(t)) if bits_ == 16 else paged.e4m3_to_f64(t.contiguous().view(torch.uint8).cpu().numpy())
                  for t in (c["k"], c["v"])]
        scales = [None if t is None else t.cpu().numpy() for t in (c["k_scale"], c["v_scale"])]
        ref = paged.decode(oracle.bf16_to_f64(bits(c["q"])), *values, c["table"].cpu().numpy(), c["pos"].cpu().numpy(), 0, 0.1, *scales)
        r = check.compare(bits(got), ref, check.TOL_FP32_P)
        assert r["ok"], r


@pytest.mark.parametrize("d, hq", [(128, 1), (256, 16)])
def test_as_many_rows_as_a_call_takes(wa, d, hq):
    """65,535 sequences, most of them over the same few pages: those of a row are what the row alone gives."""
    rows, page = 65535, 16
    gen = torch.Generator(device="cuda").manual_seed(79)
    k, v = (torch.randn((9, page, 1, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in "kv")
    q = torch.randn((rows, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.randint(0, 9, (rows, 2), generator=gen, device="cuda").int()
    pos = torch.randint(-1, 2 * page, (rows,), generator=gen, device="cuda").int()
    ws = torch.empty(wa.paged_decode_ws_bytes(rows, hq, 1, d, page, 2), dtype=torch.uint8, device="cuda")
    out = wa.paged_decode(q, k, v, table, pos, scale=0.1, ws=ws)
    assert wa.status(ws) == 0
    some = torch.tensor([0, 1, 255, 256, 63 * 1000, 65279, 65280, 65534], device="cuda")
    assert _same(out[some], wa.paged_decode(q[some], k, v, table[some], pos[some], scale=0.1))
    assert (out[pos == -1] == 0).all() and (out[pos >= 0].flatten(1) != 0).any(1).all()
