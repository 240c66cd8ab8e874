"""Append to a paged cache on the GPU against its definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from _util import bits, ensure_built
from oracle import check, paged
from test_rope_gpu import TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def pool(count, page, hkv, d, kind, heads_first, joint):
    """Keys and values as [count, page, hkv, d] views, all bits set to a pattern that is kept where nothing is written."""
    shape = (hkv, page, d) if heads_first else (page, hkv, d)
    one = torch.empty((count, 2, *shape), dtype=kind, device="cuda")
    both = [one[:, 0], one[:, 1]] if joint else [torch.empty((count, *shape), dtype=kind, device="cuda") for _ in "kv"]
    for t in both:
        t.copy_(torch.full((), 1.75, device="cuda"))
    return [t.transpose(1, 2) if heads_first else t for t in both]


def raw(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


CASES = [
    dict(rows=1, chunk=1, hq=16, hkv=8, d=256, page=16, dims=256),
    dict(rows=5, chunk=1, hq=3, hkv=3, d=128, page=32, dims=64, layout="interleaved", bits=8),
    dict(rows=3, chunk=37, hq=32, hkv=2, d=128, page=16, dims=128, bits=8, heads_first=True),
    dict(rows=4, chunk=61, hq=6, hkv=2, d=256, page=64, dims=48, layout="interleaved", joint=True),
    dict(rows=2, chunk=300, hq=8, hkv=8, d=128, page=256, dims=0, heads_first=True, joint=True),
    dict(rows=2, chunk=5, hq=5, hkv=1, d=256, page=128, dims=0, bits=8),
    dict(rows=70, chunk=40, hq=2, hkv=1, d=128, page=16, dims=128),       # more tokens than the status block takes
]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_append(wa, c):
    c = dict(dict(layout="half", bits=16, heads_first=False, joint=False), **c)
    rows, chunk, hq, hkv, d, page = (c[x] for x in ("rows", "chunk", "hq", "hkv", "d", "page"))
    rng = np.random.default_rng(rows * 100 + chunk)
    start = rng.integers(0, 1000, rows)
    pos = np.concatenate([p + np.arange(chunk) for p in start]).astype(np.int32)
    row = np.repeat(np.arange(rows), chunk).astype(np.int32)
    shuffle = rng.permutation(len(pos)) if chunk > 1 else np.arange(len(pos))
    pos, row = pos[shuffle], row[shuffle]
    most = (1000 + chunk) // page + 2
    ids = rng.permutation(rows * most + 3)
    table = ids[:rows * most].reshape(rows, most).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    src = torch.randn((len(pos), (hq + 2 * hkv) * d + 8), generator=gen, device="cuda").to(torch.bfloat16)
    kind = torch.float8_e4m3fn if c["bits"] == 8 else torch.bfloat16
    k, v = pool(len(ids), page, hkv, d, kind, c["heads_first"], c["joint"])
    before = raw(k), raw(v)
    scales = [torch.rand(hkv, generator=gen, device="cuda") * 0.1 + 0.001 if c["bits"] == 8 else None for _ in "kv"]
    inv = (10000.0 ** (-torch.arange(0, c["dims"], 2) / c["dims"])).float().cuda() if c["dims"] else None
    q = torch.full((len(pos), hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = wa.paged_append(src, torch.from_numpy(pos).cuda(), q, k, v, torch.from_numpy(table).cuda(),
                         row=None if chunk == 1 else torch.from_numpy(row).cuda(), inv_freq=inv, layout=c["layout"],
                         factor=0.75, k_scale=scales[0], v_scale=scales[1])
    assert wa.status(ws) == 0
    x = oracle.bf16_to_f64(bits(src))[:, :(hq + 2 * hkv) * d].reshape(len(pos), hq + 2 * hkv, d)
    cpu = [None if s is None else s.cpu().numpy() for s in scales]
    q_ref, q_size, places = paged.append(x, pos, row, hq, hkv, table, page, None if inv is None else inv.cpu().numpy(),
                                         c["layout"], 0.75, *cpu)
    r = check.compare(bits(q), q_ref, TOL * q_size.ravel())
    assert r["ok"], r
    got_k, got_v = raw(k), raw(v)
    assert len(places) == len(pos)
    at, slot = (np.array([p[i] for p in places]) for i in (0, 1))
    k_ref, k_size, v_ref = (np.stack([p[i] for p in places]) for i in (2, 3, 4))
    gk, gv = got_k[at, slot], got_v[at, slot]
    if c["bits"] == 16:
        r = check.compare(gk.view(np.uint16), k_ref, TOL * k_size.ravel())
        assert r["ok"], r
        assert np.array_equal(gv.view(np.uint16), oracle.f64_to_bf16(v_ref))
    else:
        # before its rounding to 8 bits a key also has the quotient's (2^-24 of it); a value has that alone, which can
        # matter where it lies next to the middle of two neighbours
        tol = TOL * k_size + 2.0 ** -23 * np.abs(k_ref)
        lo, hi = (paged.e4m3_to_f64(paged.f64_to_e4m3(k_ref + s * tol)) for s in (-1, 1))
        gk = paged.e4m3_to_f64(gk)
        assert ((lo <= gk) & (gk <= hi)).all()
        once = (x[:, hq + hkv:].astype(np.float32) / cpu[1][:, None].astype(np.float32))
        assert np.array_equal(gv & 0x7F, paged.f64_to_e4m3(once.astype(np.float64)) & 0x7F)
        assert np.array_equal(gv >> 7, np.signbit(once).astype(np.uint8))
    # every other slot as it was
    for got, was in ((got_k, before[0]), (got_v, before[1])):
        got[at, slot] = was[at, slot]
        assert np.array_equal(got, was)


@pytest.mark.parametrize("n", [6, 2100])
def test_tokens_that_are_left_out(wa, n):
    """Padding, positions past the table, rows that are none and pages that are none: nothing written, and reported."""
    hq, hkv, d, page = 4, 2, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    src = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, 1, 2], [3, -1, 99]], dtype=torch.int32, device="cuda")
    for place, status in [([(-1, 0)], 0), ([(-2, 0)], wa.WA_STATUS_BAD_POS), ([(48, 0)], wa.WA_STATUS_BAD_POS),
                          ([(2 ** 31 - 1, 0)], wa.WA_STATUS_BAD_POS), ([(5, 2)], wa.WA_STATUS_BAD_PAGE),
                          ([(5, -1)], wa.WA_STATUS_BAD_PAGE), ([(20, 1)], wa.WA_STATUS_BAD_PAGE),
                          ([(40, 1)], wa.WA_STATUS_BAD_PAGE),
                          ([(48, 0), (40, 1)], wa.WA_STATUS_BAD_POS | wa.WA_STATUS_BAD_PAGE)]:
        pos, row = torch.full((n,), -1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
        for i, (p, r) in enumerate(place):
            pos[1 + i], row[1 + i] = p, r
        pos[0] = 17                                        # one that is written
        k, v = pool(4, page, hkv, d, torch.bfloat16, False, False)
        q = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = wa.paged_append(src, pos.cuda(), q, k, v, table, row=row.cuda())
        assert wa.status(ws) == status, place
        assert torch.equal(k[1, 1], src[0].view(-1, d)[hq:hq + hkv]) and torch.equal(v[1, 1], src[0].view(-1, d)[hq + hkv:])
        k[1, 1] = v[1, 1] = 1.75
        assert (k == 1.75).all() and (v == 1.75).all(), place
        assert torch.equal(q[0], src[0].view(-1, d)[:hq])
        for i, (p, r) in enumerate(place):                 # a query whose position is good is handed on
            good = 0 <= p < 48
            assert torch.equal(q[1 + i], src[1 + i].view(-1, d)[:hq]) if good else (q[1 + i] == 7.0).all()
        assert (q[1 + len(place):] == 7.0).all()


def test_values_past_the_8_bit_range(wa):
    """448 is the largest; NaN stays NaN."""
    x = torch.tensor([0.0, 448.0, 464.0, 1e30, -1e30, float("inf"), float("-inf"), float("nan")] * 16, device="cuda")
    src = torch.cat([x, x, x]).to(torch.bfloat16).view(1, 3 * 128)
    k, v = pool(1, 16, 1, 128, torch.float8_e4m3fn, False, False)
    q = torch.empty((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    wa.paged_append(src, zero[0], q, k, v, zero)
    for t in (k, v):
        got = t[0, 0, 0, :8].float().tolist()
        assert got[:7] == [0.0, 448.0, 448.0, 448.0, -448.0, 448.0, -448.0] and np.isnan(got[7])


def test_queries_in_place_and_a_graph(wa):
    """The query heads turned where they are, and a captured step that replays with new positions."""
    n, hq, hkv, d, page = 24, 8, 4, 128, 32
    gen = torch.Generator(device="cuda").manual_seed(4)
    src = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.randperm(n * 4, generator=torch.Generator().manual_seed(5)).int().view(n, 4).cuda()
    inv, _ = wa.rope_frequencies(d, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")

    def step(x, q):
        k, v = pool(4 * n, page, hkv, d, torch.bfloat16, False, False)
        wa.paged_append(x, pos, q, k, v, table, inv_freq=inv)
        return q, k, v

    want = step(src, torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda"))
    again = src.clone()
    got = step(again, again[:, :hq * d].view(n, hq, d))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(again[:, hq * d:], src[:, hq * d:])
    q = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    k, v = pool(4 * n, page, hkv, d, torch.bfloat16, False, False)
    ws, g = torch.empty(256, dtype=torch.uint8, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wa.paged_append(src, pos, q, k, v, table, inv_freq=inv, ws=ws)
    pos.add_(40)
    g.replay()
    torch.cuda.synchronize()
    want = step(src, torch.empty_like(q))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, want[2]) and wa.status(ws) == 0
