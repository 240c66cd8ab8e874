"""Paged decode of many rows: units given out by the counter, several launches and joins, rows that are computed again."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import wa_synth
from _util import bits, ensure_built
from oracle import check
from test_paged_decode_gpu import TOL, call, reference, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def workspace(wa, c, hq):
    pages, page, hkv, d = c["k"].shape
    return torch.full((wa.paged_decode_ws_bytes(*c["table"].shape[:1], hq, hkv, d, page, c["table"].shape[1], c["win"], c["k"].dtype),), 255,
                      dtype=torch.uint8, device="cuda")


def of_rows(c, rows):
    """The case of some rows over a pool of their own pages alone (a large pool takes long in 64 bits)."""
    table = c["table"][rows]
    live = (table >= 0) & (table < c["k"].shape[0])
    ids, at = torch.unique(table[live], return_inverse=True)
    new = torch.full_like(table, -1)
    new[live] = at.int()
    own = {x: c[x].view(torch.uint8)[ids.long()].view(c[x].dtype) for x in "kv"}
    return dict(c, **own, q=c["q"][rows], table=new, pos=c["pos"][rows])


@pytest.mark.parametrize("rows, hq, hkv, d, page, win, length, bits_", [
    (150, 32, 16, 128, 16, 200, 700, 16),        # windows that begin inside a tile, in jobs
    (100, 16, 16, 256, 64, 333, 900, 16),
    (130, 32, 16, 128, 32, 500, 2000, 8),
    (90, 60, 4, 128, 16, 1500, 4000, 16),        # groups of 15 heads
    (300, 24, 2, 256, 16, 3000, 3300, 8),        # more rows than a launch, of 12 heads
    (260, 32, 2, 256, 128, 700, 1500, 16),       # five launches
    (600, 16, 8, 128, 16, 40, 300, 16),          # three
], ids=str)
def test_windows_bad_pages_and_bad_positions(wa, rows, hq, hkv, d, page, win, length, bits_):
    """Entries before the window are -1 (paged_case), one entry that is needed names no page and one position lies past the table,
    in rows of different launches: the oracle's values, the exact status, and the rest as it was."""
    lengths = [0 if r % 19 == 7 else max(1, length - 11 * (r % 23)) for r in range(rows)]
    c = wa_synth.paged_case(lengths, hq, hkv, d, page, seed=90, win=win, bits=bits_, device="cuda", outside="keep", peaked=False)
    ws = workspace(wa, c, hq)
    out = call(wa, c, 0.3, ws=ws)
    assert wa.status(ws) == 0
    some = [0, 7, rows // 3, rows // 2, rows - 1]
    r = check.compare(bits(out[some]), reference(of_rows(c, some), 0.3), TOL)
    assert r["ok"], r
    for i in some:
        one = dict(c, q=c["q"][i:i + 1], table=c["table"][i:i + 1], pos=c["pos"][i:i + 1])
        assert same(call(wa, one, 0.3)[0], out[i]), i
    for bad_entry, bad_pos in ((True, False), (False, True), (True, True)):
        for entry, place in ((rows - 2, 1), (2, rows - 3)):
            x = dict(c, table=c["table"].clone(), pos=c["pos"].clone())
            touched = []
            if bad_entry:
                x["table"][entry, (lengths[entry] - 1) // page] = c["k"].shape[0] + 5
                touched.append(entry)
            if bad_pos:
                x["pos"][place] = -7
                touched.append(place)
            got = call(wa, x, 0.3, ws=ws)
            assert wa.status(ws) == (wa.WA_STATUS_BAD_PAGE if bad_entry else 0) | (wa.WA_STATUS_BAD_POS if bad_pos else 0)
            r = check.compare(bits(got[touched]), reference(of_rows(x, touched), 0.3), TOL)
            assert r["ok"], r
            rest = [i for i in range(rows) if i not in touched]
            assert same(got[rest], out[rest])
    assert same(call(wa, c, 0.3, ws=ws), out) and wa.status(ws) == 0


@pytest.mark.parametrize("rows, hq, hkv, d, bits_", [(40, 8, 2, 128, 16), (20, 16, 1, 256, 16), (33, 8, 1, 256, 8), (330, 4, 2, 128, 16)], ids=str)
def test_non_finite_values_among_many_rows(wa, rows, hq, hkv, d, bits_):
    """From 256 (row, head) pairs on a warp joins a row's head, and its block computes again what is not finite: NaN and infinite
    keys, values and queries in some rows, as float64 has them, and every other row's bits as without them."""
    lengths = [(300, 40, 700, 129, 0)[r % 5] for r in range(rows)]
    c = wa_synth.paged_case(lengths, hq, hkv, d, 16, seed=91, bits=bits_, device="cuda", outside="keep")
    assert rows * hq >= 256
    clean = call(wa, c)
    c = dict(c, q=c["q"].clone(), k=c["k"].clone(), v=c["v"].clone())

    def put(t, r, at, g, e, x):
        t[int(c["table"][r, at // 16]), at % 16, g, e] = torch.tensor(x, device="cuda").to(t.dtype)

    inf, nan = float("inf"), float("nan")
    touched = [0, 1, 2, 6, 8, 10, 11, 12, rows - 2, rows - 6]
    put(c["k"], 0, 170, 0, 3, nan)
    put(c["v"], 1, 39, hkv - 1, 5, nan)
    if bits_ == 16:
        put(c["v"], 2, 650, 0, 0, inf)
        put(c["v"], 2, 0, 0, d - 1, -inf)
        put(c["k"], 6, 5, hkv - 1, 7, inf)
        put(c["v"], 8, 100, 0, 1, inf)
        put(c["v"], 8, 101, 0, 1, -inf)
    c["q"][10, 1, 0] = inf
    c["q"][11, hq - 1, 5] = nan
    c["q"][12, 0] *= 1e30
    put(c["v"], rows - 2, 0, 0, 64, nan)
    c["q"][rows - 6, 2] *= -1e30
    out = call(wa, c)
    r = check.compare(bits(out[touched]), reference(of_rows(c, touched), 1.0), TOL)
    assert r["ok"], r
    rest = [i for i in range(rows) if i not in touched]
    assert same(out[rest], clean[rest])
    for i in touched:                             # the other join gives the same
        one = dict(c, q=c["q"][i:i + 1], table=c["table"][i:i + 1], pos=c["pos"][i:i + 1])
        assert np.array_equal(bits(call(wa, one)[0]), bits(out[i])), i
