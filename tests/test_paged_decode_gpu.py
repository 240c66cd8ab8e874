"""Decode over a paged cache on the GPU against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import wa_synth
from _util import bits, ensure_built
from oracle import check, paged

pytestmark = pytest.mark.gpu

# Where the outputs may lie: the tolerance of fp32 probabilities that the other decode forms are held to.  What P loses in
# its parts is less: two bf16 parts 2^-17 of a weight, three e4m3 parts 2^-12, of values of up to 4.5.
TOL = check.TOL_FP32_P


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def stored(t):
    """A pool's values as float64."""
    t = t.contiguous()
    return oracle.bf16_to_f64(bits(t)) if t.dtype == torch.bfloat16 else paged.e4m3_to_f64(t.view(torch.uint8).cpu().numpy())


def reference(c, scale, rows=None):
    rows = range(len(c["pos"])) if rows is None else rows
    idx = list(rows)
    return paged.decode(oracle.bf16_to_f64(bits(c["q"]))[idx], stored(c["k"]), stored(c["v"]), c["table"].cpu().numpy()[idx],
                        c["pos"].cpu().numpy()[idx], c["win"], scale,
                        *[None if c[s] is None else c[s].cpu().numpy() for s in ("k_scale", "v_scale")])


def call(wa, c, scale=1.0, **kw):
    return wa.paged_decode(c["q"], c["k"], c["v"], c["table"], c["pos"], win=c["win"], scale=scale, k_scale=c["k_scale"],
                           v_scale=c["v_scale"], **kw)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


CASES = [
    # lengths about the tile of 128 keys and the page, an empty sequence among them
    dict(lengths=[1, 2, 16, 17, 0, 127, 128, 129, 255, 257], hq=8, hkv=4, d=128, page=16),
    dict(lengths=[300], hq=16, hkv=8, d=256, page=16),
    dict(lengths=[700, 33, 1025], hq=24, hkv=8, d=128, page=64, scale=0.0883883),
    dict(lengths=[5000, 1, 2049], hq=16, hkv=1, d=256, page=128, heads_first=True),
    dict(lengths=[4096, 130], hq=5, hkv=1, d=128, page=256, joint=True, most=64),
    dict(lengths=[3, 900], hq=4, hkv=4, d=256, page=32, heads_first=True, joint=True),
    dict(lengths=[1, 50, 100, 101, 3000], hq=32, hkv=4, d=128, page=16, win=100),
    dict(lengths=[1500, 40, 2000], hq=32, hkv=16, d=256, page=64, win=1024),
    dict(lengths=[20, 4000], hq=12, hkv=1, d=128, page=256, win=1),
    dict(lengths=[0, 0], hq=4, hkv=2, d=128, page=16),
    dict(lengths=[40] * 600, hq=2, hkv=1, d=128, page=16),
    # 8-bit pages
    dict(lengths=[1, 15, 16, 129, 2500, 0, 511], hq=32, hkv=4, d=128, page=16, bits=8, scale=0.0883883),
    dict(lengths=[40, 6000], hq=16, hkv=1, d=256, page=64, bits=8, heads_first=True),
    dict(lengths=[333, 1000], hq=6, hkv=2, d=256, page=128, bits=8, joint=True, win=700),
    dict(lengths=[2222, 5], hq=3, hkv=3, d=128, page=256, bits=8, heads_first=True, joint=True),
    dict(lengths=[129, 4001], hq=24, hkv=2, d=256, page=32, bits=8),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: ",".join(f"{k}={v if k != 'lengths' else len(v)}" for k, v in c.items()))
def test_against_the_oracle(wa, c):
    c = dict(c)
    scale = c.pop("scale", 1.0)
    x = wa_synth.paged_case(seed=len(c["lengths"]) + c["hq"], device="cuda", **c)
    ws = torch.empty(wa.paged_decode_ws_bytes(len(c["lengths"]), c["hq"], c["hkv"], c["d"], c["page"], x["table"].shape[1],
                                              c.get("win", 0), x["k"].dtype), dtype=torch.uint8, device="cuda")
    out = torch.full_like(x["q"], 9.0)
    assert call(wa, x, scale, out=out, ws=ws) is out
    r = check.compare(bits(out), reference(x, scale), TOL)
    assert r["ok"], r
    assert wa.status(ws) == 0


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("scale", [-0.5, 0.0, 4.0])
def test_scales_of_any_sign(wa, scale, bits_):
    c = wa_synth.paged_case([260, 1, 77], 8, 2, 128, 32, seed=41, bits=bits_, device="cuda")
    if bits_ == 8:
        c["k_scale"][1] *= -1
        c["v_scale"][0] *= -1
    r = check.compare(bits(call(wa, c, scale)), reference(c, scale), TOL)
    assert r["ok"], r


@pytest.mark.parametrize("bits_, d", [(16, 128), (16, 256), (8, 128), (8, 256)])
def test_equal_weights_give_the_mean(wa, bits_, d):
    """All keys zero and whole-number values: a mean over a power of two of keys is exact before its one rounding."""
    c = wa_synth.paged_case([4096, 256, 1], 8, 2, d, 64, seed=42, bits=bits_, device="cuda", peaked=False)
    gen = torch.Generator(device="cuda").manual_seed(43)
    c["k"].copy_(torch.zeros((), device="cuda"))
    c["v"].copy_(torch.randint(-8, 9, c["v"].shape, generator=gen, device="cuda").float())
    c["k_scale"] = c["v_scale"] = None
    got, ref = bits(call(wa, c)), reference(c, 1.0)
    assert np.array_equal(got, oracle.f64_to_bf16(ref))


@pytest.mark.parametrize("bits_", [16, 8])
def test_a_rows_bits_are_its_own(wa, bits_):
    """Alone, in another batch, out of other pages, of another table, the same bits."""
    lengths = [900, 5, 3000, 128, 0, 2047]
    c = wa_synth.paged_case(lengths, 16, 2, 128, 16, seed=44, bits=bits_, device="cuda", outside="keep")
    want = call(wa, c)
    for r in range(len(lengths)):
        one = dict(c, q=c["q"][r:r + 1], table=c["table"][r:r + 1], pos=c["pos"][r:r + 1])
        assert same(call(wa, one)[0], want[r]), r
    turn = torch.tensor([3, 1, 5, 0, 2, 4], device="cuda")
    moved = torch.randperm(c["k"].shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    back = torch.empty_like(moved)
    back[moved] = torch.arange(len(moved), device="cuda")
    table = torch.where(c["table"] < 0, 7, back[c["table"].long().clamp_min(0)]).int()[turn]
    wide = torch.full((6, table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    pick = moved.cpu() if bits_ == 8 else moved
    k, v = (t.view(torch.uint8).cpu()[pick].cuda().view(t.dtype) if bits_ == 8 else t[pick] for t in (c["k"], c["v"]))
    got = call(wa, dict(c, q=c["q"][turn], k=k, v=v, table=wide[:, :table.shape[1] + 4], pos=c["pos"][turn]))
    assert same(got, want[turn])


@pytest.mark.parametrize("d, hq, hkv", [(128, 16, 2), (256, 24, 4)])
def test_a_rows_bits_in_batches_of_many_rows(wa, d, hq, hkv):
    """A row of many spans alone, and among enough rows that others join its spans."""
    lengths = [20000, 700, 0, 2500] + [33] * 60
    c = wa_synth.paged_case(lengths, hq, hkv, d, 64, seed=53, device="cuda", outside="keep")
    want = call(wa, c)
    for r in (0, 1, 2, 3, 63):
        one = dict(c, q=c["q"][r:r + 1], table=c["table"][r:r + 1], pos=c["pos"][r:r + 1])
        assert same(call(wa, one)[0], want[r]), r
    r = check.compare(bits(want[:5]), reference(c, 1.0, rows=range(5)), TOL)
    assert r["ok"], r


@pytest.mark.parametrize("rows, hq, hkv, d, length, bits_", [
    (48, 32, 16, 128, 300, 16),         # more units than the CTAs take in turn: short ones, given out by jobs,
    (40, 64, 16, 256, 260, 16),
    (64, 32, 16, 128, 900, 8),
    (24, 32, 8, 128, 8000, 16),         # and long ones, one by one
    (30, 16, 2, 256, 20000, 8),
    (70, 16, 1, 256, 140, 16),          # and more rows than one launch takes
    (300, 8, 4, 128, 140, 8),
], ids=str)
def test_large_batches(wa, rows, hq, hkv, d, length, bits_):
    """Rows of like lengths, some empty: sampled rows against the oracle, and alone."""
    lengths = [0 if r % 17 == 5 else max(1, length - 7 * (r % 13)) for r in range(rows)]
    c = wa_synth.paged_case(lengths, hq, hkv, d, 64, seed=54, bits=bits_, device="cuda", outside="keep", peaked=False)
    out = call(wa, c)
    some = [0, 5, rows // 2, rows - 1]
    r = check.compare(bits(out[some]), reference(c, 1.0, rows=some), TOL)
    assert r["ok"], r
    for i in some:
        one = dict(c, q=c["q"][i:i + 1], table=c["table"][i:i + 1], pos=c["pos"][i:i + 1])
        assert same(call(wa, one)[0], out[i]), i
    for _ in range(3):                  # whoever takes which unit
        assert same(call(wa, c), out)


def test_parts_of_a_pool(wa):
    """Some heads, some slots and some pages of a larger pool."""
    c = wa_synth.paged_case([300, 64], 8, 2, 128, 16, seed=55, device="cuda")
    pages = c["k"].shape[0]
    pool = torch.full((2 * pages, 32, 5, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = pool[::2, :16, 3:], pool[1::2, 16:, 1:3]
    k.copy_(c["k"])
    v.copy_(c["v"])
    want = call(wa, c)
    assert same(call(wa, dict(c, k=k, v=v)), want)


def test_the_widest_window(wa):
    c = wa_synth.paged_case([300, 64], 8, 2, 128, 16, seed=56, device="cuda")
    want = call(wa, c)
    for win in (300, 2 ** 31 - 1):
        assert wa.paged_decode_ws_bytes(2, 8, 2, 128, 16, c["table"].shape[1], win) == \
            wa.paged_decode_ws_bytes(2, 8, 2, 128, 16, c["table"].shape[1])
        assert same(call(wa, dict(c, win=win)), want)


def test_strided_queries_and_outputs_and_shared_pages(wa):
    """Queries inside projection rows, outputs inside a wider buffer, and two sequences with a common prefix."""
    c = wa_synth.paged_case([200, 200], 8, 4, 128, 64, seed=45, device="cuda")
    c["table"][1, :3] = c["table"][0, :3]
    wide = torch.zeros((2, 16 * 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :8 * 128] = c["q"].view(2, -1)
    c["q"] = wide[:, :8 * 128].view(2, 8, 128)
    buf = torch.full((2, 10, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    call(wa, c, out=buf[:, 1:9])
    r = check.compare(bits(buf[:, 1:9]), reference(c, 1.0), TOL)
    assert r["ok"], r
    assert (buf[:, 0] == 3.0).all() and (buf[:, 9] == 3.0).all()


@pytest.mark.parametrize("bits_", [16, 8])
def test_bad_positions_and_pages(wa, bits_):
    """Clamped, or read as zeros, and reported; a good call on the same workspace afterwards is clean."""
    c = wa_synth.paged_case([100, 64, 150], 4, 2, 128, 16, seed=46, bits=bits_, device="cuda", most=10, outside="keep")
    ws = torch.empty(wa.paged_decode_ws_bytes(3, 4, 2, 128, 16, 10, 0, c["k"].dtype), dtype=torch.uint8, device="cuda")
    good = call(wa, c, ws=ws)
    assert wa.status(ws) == 0
    for p, t, status in [([99, 63, -2], None, wa.WA_STATUS_BAD_POS), ([99, -2 ** 31, 149], None, wa.WA_STATUS_BAD_POS),
                         ([99, 63, 149], (0, 3, -1), wa.WA_STATUS_BAD_PAGE),
                         ([99, 63, 149], (2, 9, 2 ** 31 - 1), wa.WA_STATUS_BAD_PAGE),
                         ([99, 63, 149], (2, 0, c["k"].shape[0]), wa.WA_STATUS_BAD_PAGE)]:
        x = dict(c, pos=torch.tensor(p, dtype=torch.int32, device="cuda"), table=c["table"].clone())
        if t:
            x["table"][t[0], t[1]] = t[2]
        got = call(wa, x, ws=ws)
        assert wa.status(ws) == status, (p, t)
        r = check.compare(bits(got), reference(x, 1.0), TOL)
        assert r["ok"], r
    x = dict(c, pos=torch.tensor([99, 63, 160], dtype=torch.int32, device="cuda"))    # the table's last position is 159
    call(wa, x, ws=ws)
    assert wa.status(ws) == wa.WA_STATUS_BAD_POS
    assert same(call(wa, c, ws=ws), good) and wa.status(ws) == 0


@pytest.mark.parametrize("d, hq, hkv", [(128, 8, 2), (256, 16, 1)])
def test_non_finite_values(wa, d, hq, hkv):
    """As float64 has them: a NaN key, infinite keys of both signs, infinite and NaN values, an infinite query."""
    lengths = [300, 300, 1000, 300, 40, 300, 700]
    c = wa_synth.paged_case(lengths, hq, hkv, d, 16, seed=47, device="cuda")

    def put(t, r, at, g, e, x):
        t[int(c["table"][r, at // 16]), at % 16, g, e] = x

    put(c["k"], 0, 170, 0, 3, float("nan"))
    put(c["k"], 1, 5, hkv - 1, 7, float("inf"))
    put(c["v"], 2, 999, 0, 0, float("inf"))
    put(c["v"], 2, 0, 0, d - 1, float("-inf"))
    put(c["v"], 3, 299, hkv - 1, 5, float("nan"))
    put(c["v"], 6, 350, 0, 1, float("inf"))
    put(c["v"], 6, 351, 0, 1, float("-inf"))
    c["q"][4, 1, 0] = float("inf")
    c["q"][5, 0] *= 1e30              # scores of about 1e31: the softmax is a maximum
    out = call(wa, c)
    r = check.compare(bits(out), reference(c, 1.0), TOL)
    assert r["ok"], r


def test_non_finite_8_bit_values(wa):
    c = wa_synth.paged_case([300, 300, 40], 8, 2, 128, 16, seed=48, bits=8, device="cuda")
    nan = torch.tensor(float("nan"), device="cuda").to(torch.float8_e4m3fn)
    c["k"][int(c["table"][0, 4]), 3, 0, 9] = nan
    c["v"][int(c["table"][1, 18]), 11, 1, 100] = nan
    c["q"][2, 5, 7] = float("-inf")
    c["q"][2, 1] *= 1e30
    c["q"][2, 2] *= 1e-30
    r = check.compare(bits(call(wa, c)), reference(c, 1.0), TOL)
    assert r["ok"], r


def test_a_long_row_and_far_pages(wa):
    """Many spans of one row; the last pages of a pool of more than 2^32 elements."""
    n, page, hkv, d = 70001, 64, 1, 128
    c = wa_synth.paged_case([n], 8, hkv, d, page, seed=49, device="cuda")
    r = check.compare(bits(call(wa, c)), reference(c, 1.0), TOL)
    assert r["ok"], r
    pages = 2 ** 32 // (page * 8 * d) + 40
    k = torch.empty((pages, page, 8, d), dtype=torch.bfloat16, device="cuda")
    c = wa_synth.paged_case([500], 16, 8, d, page, seed=50, device="cuda")
    live = c["k"].shape[0]
    far = dict(c, k=k, v=k, table=(c["table"] + pages - live).int())
    k[-live:] = c["k"]
    near_ = dict(c, v=c["k"])
    assert same(call(wa, far), call(wa, near_))


def test_streams_and_graphs(wa):
    """Two calls at once on two streams, and a captured step that replays with a longer sequence and other pages."""
    a = wa_synth.paged_case([3000, 10, 777], 32, 4, 128, 16, seed=51, device="cuda", outside="keep", most=300)
    b = wa_synth.paged_case([500] * 8, 16, 8, 256, 64, seed=52, device="cuda", outside="keep")
    want = call(wa, a), call(wa, b)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [call(wa, c, stream=x) for c, x in zip((a, b), s)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])
    out, ws = torch.empty_like(a["q"]), torch.empty(wa.paged_decode_ws_bytes(3, 32, 4, 128, 16, 300), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(wa, a, out=out, ws=ws)
    for step in range(3):
        a["pos"].copy_(torch.tensor([2999 - 100 * step, 9, 776 - step], dtype=torch.int32))
        a["q"].copy_(torch.roll(a["q"], 1, dims=1))
        g.replay()
        torch.cuda.synchronize()
        assert same(out, call(wa, a)) and wa.status(ws) == 0
