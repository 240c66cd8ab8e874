"""The status word of appends of more tokens than one block checks: every bad token is reported wherever it stands, and a good
call on the same workspace is clean afterwards."""
from __future__ import annotations

import pytest
import torch

from _util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("n, hq, hkv, d, kind", [(1024, 1, 1, 128, torch.bfloat16), (1025, 1, 1, 128, torch.bfloat16), (5000, 8, 1, 128, torch.bfloat16),
                                                 (3333, 32, 8, 128, torch.float8_e4m3fn), (2000, 6, 3, 256, torch.bfloat16)], ids=str)
def test_a_bad_token_anywhere(wa, n, hq, hkv, d, kind):
    page, rows = 16, 7
    most = (n // rows + 1) // page + 1
    gen = torch.Generator(device="cuda").manual_seed(84)
    src = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.randperm(rows * most, generator=torch.Generator().manual_seed(85)).int().view(rows, most).cuda()
    row = (torch.arange(n) % rows).int().cuda()
    pos = (torch.arange(n) // rows).int().cuda()
    k, v = (torch.zeros((rows * most, page, hkv, d), device="cuda").to(kind) for _ in "kv")
    q = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")        # whatever a workspace holds before
    raw = lambda t: t.view(torch.uint8).reshape(rows * most * page, -1)   # noqa: E731
    slot = table.long()[row.long(), pos.long() // page] * page + pos.long() % page

    def run(p, r):
        k.view(torch.uint8).zero_(), v.view(torch.uint8).zero_(), q.zero_()
        wa.paged_append(src, p, q, k, v, table, row=r, ws=ws)
        return wa.status(ws)

    assert run(pos, row) == 0
    want = q.clone(), raw(k)[slot].clone(), raw(v)[slot].clone()
    assert torch.equal(want[0], src.view(n, -1, d)[:, :hq])
    for at in (0, 1, n // 2, n - 2, n - 1):
        for bad, status in ((dict(pos=-2), wa.WA_STATUS_BAD_POS), (dict(pos=most * page), wa.WA_STATUS_BAD_POS), (dict(row=rows), wa.WA_STATUS_BAD_PAGE),
                            (dict(row=-1), wa.WA_STATUS_BAD_PAGE), (dict(pos=-1), 0)):
            p, r = pos.clone(), row.clone()
            p[at], r[at] = bad.get("pos", p[at]), bad.get("row", r[at])
            assert run(p, r) == status, (at, bad)
            # that token's place is as it was, every other token's is written
            assert (raw(k)[slot[at]] == 0).all() and (raw(v)[slot[at]] == 0).all()
            rest = torch.arange(n, device="cuda") != at
            assert torch.equal(raw(k)[slot[rest]], want[1][rest]) and torch.equal(raw(v)[slot[rest]], want[2][rest])
            assert torch.equal(q[rest], want[0][rest]) and torch.equal(q[at], want[0][at] if "row" in bad else torch.zeros_like(q[at]))
    p, r = pos.clone(), row.clone()
    p[3], r[n - 4] = 2 ** 31 - 1, 2 ** 31 - 1
    assert run(p, r) == wa.WA_STATUS_BAD_POS | wa.WA_STATUS_BAD_PAGE
    assert run(torch.full_like(pos, -5), row) == wa.WA_STATUS_BAD_POS and not q.any()     # all of them
    assert run(pos, row) == 0 and torch.equal(q, want[0])


def test_a_captured_append_of_many_tokens(wa):
    """Replays clear and report anew each time, one after another and two graphs of workspaces of their own at once."""
    n, rows, hq, hkv, d, page, most = 2100, 3, 4, 2, 128, 16, 44
    gen = torch.Generator(device="cuda").manual_seed(86)
    src = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device="cuda").to(torch.bfloat16)
    row = (torch.arange(n) % rows).int().cuda()
    sets = []
    for i in range(2):
        table = torch.randperm(rows * most, generator=torch.Generator().manual_seed(i)).int().view(rows, most).cuda()
        s = dict(pos=(torch.arange(n) // rows).int().cuda(), table=table, q=torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda"),
                 k=torch.zeros((rows * most, page, hkv, d), dtype=torch.bfloat16, device="cuda"),
                 v=torch.zeros((rows * most, page, hkv, d), dtype=torch.bfloat16, device="cuda"),
                 ws=torch.full((256,), 255, dtype=torch.uint8, device="cuda"), g=torch.cuda.CUDAGraph(), stream=torch.cuda.Stream())
        with torch.cuda.graph(s["g"]):
            wa.paged_append(src, s["pos"], s["q"], s["k"], s["v"], table, row=row, ws=s["ws"])
        sets.append(s)
    for step in range(6):
        for i, s in enumerate(sets):
            s["pos"][17] = (5, -2, 5)[(step + i) % 3]
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["g"].replay()
        torch.cuda.synchronize()
        for i, s in enumerate(sets):
            assert wa.status(s["ws"]) == (0, wa.WA_STATUS_BAD_POS, 0)[(step + i) % 3]
            assert torch.equal(s["q"][18:], src.view(n, -1, d)[18:, :hq])
