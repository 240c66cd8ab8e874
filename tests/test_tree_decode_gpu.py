"""Tree decode on the GPU against the float64 definition.

Tolerance: the decode form's, [RN(o - 3e-3), RN(o + 3e-3)] in bf16 value order.  What the kernel may be off by
stays inside it: a score is an fp32 sum of d exact products, off by at most d 2^-24 sum|q_e k_e| (d = 256, scores
to 30: under 5e-4); a weight by that, by the exponential's 2^-22 and by the two-part P's 2^-17; the output, a mean
of values of at most about 4.5 in size, by twice that times 4.5 at worst and by far less on average.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import wa_synth
from _util import assert_parity, bits, ensure_built
from oracle import check, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def _case(rows, nodes, hq, hkv, d, win, ring, pos, **kw):
    return wa_synth.tree_case(rows, nodes, hq, hkv, d, win, ring, pos, device="cuda", **kw)


def _run(wa, c, scale=1.0, **kw):
    a = dict(n=c["n"], scale=scale)
    a.update(kw)
    return wa.tree_decode(c["q"], c["k"], c["v"], c["k_tree"], c["v_tree"], c["pos"], c["parent"], c["win"], **a)


def _ref(c, scale=1.0):
    n = None if c["n"] is None else c["n"].tolist()
    return tree.decode(bits(c["q"]), bits(c["k"]), bits(c["v"]), bits(c["k_tree"]), bits(c["v_tree"]),
                       c["pos"].tolist(), c["parent"].cpu().numpy(), c["win"], scale, n)


def _check(got, ref, c, what=""):
    n = [c["nodes"]] * c["rows"] if c["n"] is None else [min(max(x, 0), c["nodes"]) for x in c["n"].tolist()]
    for r, live in enumerate(n):
        if live:
            assert_parity(got[r, :live], ref[r, :live], check.TOL_FP32_P, f"{what} row {r}")


def _eq(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


CASES = [
    # rows, nodes, hq, hkv, d, win, ring, pos, kind, n
    (1, 1, 2, 1, 256, 0, 64, [0], "chain", None),
    (1, 1, 16, 1, 128, 0, 200, [-1], "chain", None),
    (2, 8, 16, 8, 256, 1024, 1536, [900, 40000], "random", None),
    (3, 16, 4, 2, 256, 0, 700, [699, 511, 128], "bushy", [16, 7, 1]),
    (2, 27, 6, 2, 128, 100, 111, [60, 5000], "random", [27, 13]),
    (4, 5, 3, 1, 128, 0, 130, [126, 127, 128, 129], "random", None),
    (2, 128, 2, 2, 128, 300, 300, [299, 777], "chain", None),      # the tree reaches past the window's own keys
    (1, 128, 16, 1, 256, 0, 300, [255], "random", None),
    (2, 64, 8, 1, 128, 0, 1100, [1023, 40], "bushy", None),
    (2, 40, 5, 1, 256, 17, 23, [22, 1000], "chain", [40, 33]),      # window shorter than the chain
    (2, 6, 2, 1, 128, 1, 1, [3, -1], "random", None),               # a window of one: itself alone
    (2, 9, 4, 4, 128, 0, 64, [63, -1], "flat", None),               # all nodes roots; a full linear cache
    (3, 12, 8, 2, 256, 1000, 1003, [998, 1002, 123456], "random", [0, 12, 5]),
    (1, 11, 7, 1, 128, 0, 2600, [2555], "random", None),
    (1, 3, 32, 2, 256, 2048, 2048, [9000], "chain", None),
    (2, 10, 26, 2, 128, 0, 300, [290, 13], "bushy", None),          # groups of 13: idle lanes
]


@pytest.mark.parametrize("shape", CASES, ids=lambda s: "x".join(map(str, s[:7])))
def test_parity(wa, shape):
    rows, nodes, hq, hkv, d, win, ring, pos, kind, n = shape
    c = _case(rows, nodes, hq, hkv, d, win, ring, pos, seed=rows * 1000 + nodes, kind=kind, n=n)
    ws = torch.empty(wa.tree_decode_ws_bytes(rows, nodes, hq, hkv, d, win, ring), dtype=torch.uint8, device="cuda")
    out = torch.full_like(c["q"], 7.0)
    got = _run(wa, c, out=out, ws=ws)
    assert got is out and wa.status(ws) == 0
    _check(got, _ref(c), c)
    for r, live in enumerate([] if n is None else n):      # nodes past n are left as they were
        assert (got[r, live:] == 7.0).all()


@pytest.mark.parametrize("scale", [-0.7, 0.0, 0.0625])
@pytest.mark.parametrize("d", [128, 256])
def test_scales(wa, scale, d):
    c = _case(2, 9, 4, 2, d, 0, 400, [399, 150], seed=4)
    _check(_run(wa, c, scale), _ref(c, scale), c)


@pytest.mark.parametrize("d", [128, 256])
def test_strided_nodes_and_outputs(wa, d):
    """q and v as views of one projection buffer, k_tree with nodes before rows, an output between other data."""
    rows, nodes, hq, hkv = 3, 10, 4, 2
    c = _case(rows, nodes, hq, hkv, d, 300, 320, [40, 700, 319], seed=9, n=[10, 4, 9])
    fused = torch.zeros((rows, nodes, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device="cuda")
    q = fused[:, :, :hq * d].unflatten(2, (hq, d))
    v = fused[:, :, (hq + hkv) * d:].unflatten(2, (hkv, d))
    q.copy_(c["q"])
    v.copy_(c["v_tree"])
    k = torch.zeros((nodes, rows, hkv, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    k.copy_(c["k_tree"])
    wide = torch.full((rows, nodes + 2, hq + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 1:nodes + 1, :hq]
    out = wide.as_strided((rows, nodes, hq, d), (wide.stride(0), wide.stride(1), d, 1), wide.stride(1))
    want = _run(wa, c)
    wa.tree_decode(q, c["k"], c["v"], k, v, c["pos"], c["parent"], c["win"], n=c["n"], out=out)
    for r, live in enumerate(c["n"].tolist()):
        assert _eq(out[r, :live], want[r, :live])
        assert (out[r, live:] == 3.0).all()
    assert (wide[:, 0] == 3.0).all() and (wide[:, -1] == 3.0).all() and (wide[:, :, hq] == 3.0).all()


@pytest.mark.parametrize("hkv,win,ring", [(2, 0, 5000), (1, 600, 640), (8, 2048, 2100)])
def test_bits_depend_on_the_row_alone(wa, hkv, win, ring):
    """Batch, slot, padding of the tree, and the length that a linear cache is declared with."""
    pos = [4500, 100, 4999, 777]
    c = _case(4, 20, hkv * 4, hkv, 128, win, ring, pos, seed=31, outside="keep")
    got = _run(wa, c)
    for r in (3, 0):
        one = wa.tree_decode(c["q"][r:r + 1], c["k"][r:r + 1], c["v"][r:r + 1], c["k_tree"][r:r + 1],
                             c["v_tree"][r:r + 1], c["pos"][r:r + 1], c["parent"][r:r + 1], win)
        assert _eq(one[0], got[r])
    few = wa.tree_decode(c["q"][:, :7].contiguous(), c["k"], c["v"], c["k_tree"][:, :7].contiguous(),
                         c["v_tree"][:, :7].contiguous(), c["pos"], c["parent"][:, :7].contiguous(), win)
    assert _eq(few, got[:, :7])
    some = _run(wa, c, n=torch.tensor([7, 20, 1, 13], dtype=torch.int32, device="cuda"))
    for r, live in enumerate([7, 20, 1, 13]):
        assert _eq(some[r, :live], got[r, :live])
    if win == 0:
        longer = torch.cat([c["k"], c["k"][:, :3777]], 1), torch.cat([c["v"], c["v"][:, :3777]], 1)
        assert _eq(wa.tree_decode(c["q"], *longer, c["k_tree"], c["v_tree"], c["pos"], c["parent"], 0), got)


def test_other_branches_do_not_matter(wa):
    """A node's bits stay when another branch's keys and values change; where they turn NaN or infinite, its values
    stay those of the definition.  (A masked NaN value meets a zero probability in the products, the result is NaN
    and is computed again in float64: the correctly rounded value, which the fp32 result may miss by a bf16 step.
    So the two are held to the same range and not to each other's bits.)"""
    c = _case(2, 13, 8, 2, 256, 0, 300, [255, 31], seed=12, kind="bushy")
    got = _run(wa, c)
    parents = c["parent"][0].tolist()
    off = [i for i in range(13) if 1 in tree.chain(parents, i)]       # the branch below node 1
    rest = [i for i in range(13) if i not in off]
    kt, vt = c["k_tree"].clone(), c["v_tree"].clone()
    c["k_tree"][:, off] = 50.0 * kt[:, off]
    c["v_tree"][:, off] = -3e4
    assert _eq(_run(wa, c)[:, rest], got[:, rest])
    c["k_tree"][:, off] = float("nan")
    c["v_tree"][:, off] = vt[:, off]
    assert _eq(_run(wa, c)[:, rest], got[:, rest])      # a masked key's score never enters
    c["v_tree"][:, off[0]] = float("inf")
    c["v_tree"][:, off[1:]] = float("nan")
    again = _run(wa, c)
    _check(again, _ref(c), c)
    assert torch.isfinite(again[:, rest]).all() and torch.isnan(again[:, off]).all()


@pytest.mark.parametrize("d", [128, 256])
def test_non_finite_values_follow_the_formula(wa, d):
    """NaN query, NaN key, infinite values in the cache and in the tree, a window that hides them from some nodes."""
    c = _case(3, 14, 4, 2, d, 64, 90, [200, 200, 70], seed=8, kind="chain")
    c["q"][0, 3, 1] = float("nan")
    c["k"][1, (200 - 60) % 90, 0] = float("nan")        # the first nodes see it, later ones have left it behind
    c["v"][1, 195 % 90, 1, 5] = float("inf")
    c["v"][1, 196 % 90, 1, 5] = float("-inf")
    c["v_tree"][2, 4, 0, 7] = float("-inf")
    c["k_tree"][2, 9, 1, 0] = float("inf")
    _check(_run(wa, c), _ref(c), c)


def test_large_scores(wa):
    """Scores far beyond the exponential's range (one key takes all the weight), and ties."""
    c = _case(1, 6, 2, 1, 128, 0, 600, [599], seed=2)
    c["k"].mul_(300.0)
    c["k"][0, 5] = c["k"][0, 3]
    _check(_run(wa, c), _ref(c), c)


def test_equal_keys_give_the_exact_mean(wa):
    """Every weight is 1: integer values sum exactly in fp32, so the mean is the correctly rounded quotient."""
    rows, nodes, d, ring = 2, 8, 256, 1000
    c = _case(rows, nodes, 4, 2, d, 0, ring, [999, 500], seed=5, kind="chain", outside="keep")
    for x in ("k", "k_tree"):
        c[x].zero_()
    for x in ("v", "v_tree"):
        c[x].copy_(torch.randint(-8, 9, c[x].shape, device="cuda").to(torch.bfloat16))
    got = _run(wa, c)
    for r, p in enumerate(c["pos"].tolist()):
        total = c["v"][r, :p + 1].double().sum(0) + c["v_tree"][r].double().cumsum(0)        # [nodes, hkv, d]
        count = torch.arange(p + 2, p + 2 + nodes, device="cuda")[:, None, None]
        want = (total.float() / count.float()).to(torch.bfloat16).repeat_interleave(2, 1)
        # fp32 quotient of exact integers, as O / l or O * (1 / l): one fp32 step at most before bf16
        assert (got[r].float() - want.float()).abs().le(want.float().abs() * 2 ** -8).all()
        assert (got[r] == want).float().mean() > 0.999


def test_status_bits(wa):
    c = _case(3, 6, 2, 1, 128, 0, 100, [50, 60, 70], seed=1, outside="keep")
    ws = torch.empty(wa.tree_decode_ws_bytes(3, 6, 2, 1, 128, 0, 100), dtype=torch.uint8, device="cuda")
    good = _run(wa, c)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    c["pos"] = i32(50, 100, 70)
    _run(wa, c, ws=ws)
    assert wa.status(ws) == wa.WA_STATUS_BAD_POS
    c["pos"] = i32(50, -2, 70)
    _run(wa, c, ws=ws)
    assert wa.status(ws) == wa.WA_STATUS_BAD_POS
    c["pos"] = i32(50, 60, 70)
    for bad in (6, 2, -2, 2 ** 31 - 1, -2 ** 31):
        c["parent"][1, 2] = bad
        got = _run(wa, c, ws=ws)
        assert wa.status(ws) == wa.WA_STATUS_BAD_TREE
        assert _eq(got[[0, 2]], good[[0, 2]])
        _check(got, _ref(c), c)                       # the node counts as a root
    c["parent"][1, 2] = 1
    for bad in (7, -1):
        got = _run(wa, c, n=i32(6, bad, 6), ws=ws)
        assert wa.status(ws) == wa.WA_STATUS_BAD_TREE
        assert _eq(got[[0, 2]], good[[0, 2]])
    _run(wa, c, ws=ws)
    assert wa.status(ws) == 0


def test_streams_and_graphs(wa):
    """Two streams at once with workspaces of their own; a captured call replayed on changed inputs."""
    cs = [_case(4, 12, 8, 4, 256, 512, 640, [100, 600, 5000, 641], seed=s, outside="keep") for s in (1, 2)]
    want = [_run(wa, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [_run(wa, c, stream=s) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    assert all(_eq(a, b) for a, b in zip(got, want))

    c = cs[0]
    out = torch.zeros_like(c["q"])
    ws = torch.empty(wa.tree_decode_ws_bytes(4, 12, 8, 4, 256, 512, 640), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        _run(wa, c, out=out, ws=ws, stream=streams[0])
    for step in range(3):
        c["pos"].add_(5)
        c["parent"].copy_(torch.tensor(wa_synth.draft_tree("random", 12, 50 + step), device="cuda").expand(4, 12))
        c["q"].copy_(torch.roll(c["q"], 1, dims=2))
        g.replay()
        torch.cuda.synchronize()
        assert _eq(out, _run(wa, c)) and wa.status(ws) == 0


def test_offsets_past_32_bits(wa):
    """The second row's ring starts past 2^31 elements; its nodes against a float64 product on the device."""
    rows, ring, hkv, d, nodes = 2, 280_000, 32, 128, 5
    k = torch.empty((rows, ring, hkv, d), dtype=torch.bfloat16, device="cuda").normal_(0, 0.1)
    v = torch.empty_like(k).normal_()
    q = torch.randn((rows, nodes, hkv, d), device="cuda").to(torch.bfloat16)
    kt, vt = torch.randn_like(q), torch.randn_like(q)
    pos = torch.tensor([-1, ring - 1], dtype=torch.int32, device="cuda")
    parent = torch.tensor([[-1, 0, 1, 2, 3]] * rows, dtype=torch.int32, device="cuda")
    got = wa.tree_decode(q, k, v, kt, vt, pos, parent, 0, scale=0.088)
    for h in (0, 31):
        for i in (0, 4):
            kk = torch.cat([k[1, :, h], kt[1, :i + 1, h]]).double()
            vv = torch.cat([v[1, :, h], vt[1, :i + 1, h]]).double()
            o = torch.softmax(0.088 * (kk @ q[1, i, h].double()), 0) @ vv
            assert_parity(got[1, i, h], o.cpu().numpy(), check.TOL_FP32_P)
    ref = tree.decode(bits(q[:1]), bits(k[:1, :1]), bits(v[:1, :1]), bits(kt[:1]), bits(vt[:1]), [-1],
                      parent[:1].cpu().numpy(), 0, 0.088)
    assert_parity(got[0], ref[0], check.TOL_FP32_P)
    assert np.isfinite(ref).all()


def test_rows_without_nodes(wa):
    """No row has a node: nothing is written, and a call behind it on the same workspace is not disturbed."""
    c = _case(5, 7, 4, 2, 128, 0, 1000, [-1, 0, 500, 999, 12], seed=6, outside="keep")
    ws = torch.empty(wa.tree_decode_ws_bytes(5, 7, 4, 2, 128, 0, 1000), dtype=torch.uint8, device="cuda")
    want = _run(wa, c)
    out = torch.full_like(c["q"], 7.0)
    none = torch.zeros(5, dtype=torch.int32, device="cuda")
    for _ in range(20):
        _run(wa, c, n=none, out=out, ws=ws)
        got = _run(wa, c, ws=ws)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and _eq(got, want) and wa.status(ws) == 0


def test_more_rows_than_the_plan_has_threads(wa):
    """1,100 rows of their own lengths, each as it would be alone (checked for some) and by the definition."""
    rows = 1100
    pos = [(37 * r) % 1301 - 1 for r in range(rows)]
    n = [r % 4 for r in range(rows)]
    c = _case(rows, 3, 2, 1, 128, 0, 1300, pos, seed=12, n=n, outside="keep")
    ws = torch.empty(wa.tree_decode_ws_bytes(rows, 3, 2, 1, 128, 0, 1300), dtype=torch.uint8, device="cuda")
    got = _run(wa, c, out=torch.zeros_like(c["q"]), ws=ws)
    assert wa.status(ws) == 0
    pick = [0, 1, 31, 32, 1023, 1025, 1026, 1099]
    sub = dict(c, rows=len(pick))
    for x in ("q", "k", "v", "k_tree", "v_tree", "pos", "parent", "n"):
        sub[x] = c[x][pick].contiguous()
    ref = _ref(sub)
    _check(got[pick], ref, sub)
    alone = _run(wa, sub, out=torch.zeros_like(sub["q"]))
    assert _eq(got[pick], alone)
    c["parent"][1090, 1], c["pos"][1091] = 1, 1300          # found by threads that take a second row
    c["n"][1090] = 2
    _run(wa, c, ws=ws)
    assert wa.status(ws) == wa.WA_STATUS_BAD_TREE | wa.WA_STATUS_BAD_POS


def test_two_captured_calls_replayed_at_once(wa):
    """Two graphs of several calls each, with workspaces of their own, on two streams: as the calls one by one."""
    cs = [_case(3, 20, 8, 2, 256, 0, 3000, [2999, 100, -1], seed=31, outside="keep"),
          _case(6, 33, 8, 8, 128, 700, 720, [5, 719, 720, 100000, 699, 40], seed=32, outside="keep")]
    want = [_run(wa, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[torch.zeros_like(c["q"]) for _ in range(3)] for c in cs]
    graphs = []
    torch.cuda.synchronize()
    for c, s, out in zip(cs, streams, outs):
        ws = torch.empty(wa.tree_decode_ws_bytes(c["rows"], c["nodes"], c["q"].shape[2], c["k"].shape[2], c["q"].shape[3],
                                                 c["win"], c["k"].shape[1]), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for o in out:                    # one behind another on one workspace
                _run(wa, c, out=o, ws=ws, stream=s)
        graphs.append((g, s, ws))
    for _ in range(10):
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, out, (_, _, ws) in zip(want, outs, graphs):
        assert all(_eq(o, w) for o in out) and wa.status(ws) == 0


def test_beside_the_other_tensor_core_kernels(wa):
    """A tree decode, a decode and a prompt at the same time on three streams."""
    c = _case(8, 16, 16, 2, 256, 0, 4000, [3999 - 300 * r for r in range(8)], seed=41, outside="keep")
    dc = wa_synth.decode_case(8, 16, 2, 256, 1024, 1024, [3000 + r for r in range(8)], seed=42, device="cuda")
    pc = wa_synth.prompt_case(500, 100, 8, 4, 128, 0, 600, seed=43, device="cuda")
    s = [torch.cuda.Stream() for _ in range(3)]
    calls = [lambda s: _run(wa, c, stream=s),
             lambda s: wa.decode(dc["q"], dc["k"], dc["v"], dc["pos"], 1024, 1.0, stream=s),
             lambda s: wa.prompt(pc["q"], pc["k"], pc["v"], 100, None, 0, 0.088, stream=s)]
    want = [f(torch.cuda.current_stream()) for f in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [f(x) for f, x in zip(calls, s)]
    torch.cuda.synchronize()
    assert all(_eq(a, b) for a, b in zip(got, want))
    again = _run(wa, c)                  # the ordinary call's way gives the same bits as the one with a stream
    assert _eq(again, want[0])


def test_weights_enter_the_products_within_half_a_step_of_two_parts(wa):
    """A root sees one ring key of weight 1 and itself with weight p = e^s in (1/2, 1), s a bf16 number, so scores
    are exact; the ring's value is a, the node's -b, with b near a / p, so that what is left of a - p b shows p's error.

    Tolerance, before the first run: p in two bf16 parts is off by at most 2^-18 here (the first part by half of its
    step 2^-8, so the rest is at most 2^-9 and its step 2^-17); the exponential by 2^-22 and its argument's roundings by
    less; products are exact, and each of the few fp32 sums of terms up to 2 is off by at most 2^-23 (one that cuts, at
    |terms| up to 2), 2^-21 in all.  Over l = 1 + p >= 1.5 and with b <= 4: (4 (2^-18 + 2^-21) + 2^-21) / l, the l's own
    2^-23 of a result below 2^-6, and the output's rounding: 2^-8 of its value at most."""
    rows, nodes, heads, d = 4, 128, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(17)
    s = (-0.69 * torch.rand((rows, nodes, heads), generator=gen, device="cuda")).to(torch.bfloat16)
    p = s.double().exp()
    assert p.min() > 0.5
    q = torch.zeros((rows, nodes, heads, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    kt = torch.zeros_like(q)
    kt[..., 0] = s
    a = (1.0 + torch.arange(d, device="cuda") / 128.0).to(torch.bfloat16)
    b = (a.double() / p[..., None]).to(torch.bfloat16)
    k = torch.zeros((rows, 1, heads, d), dtype=torch.bfloat16, device="cuda")
    v = a.expand(rows, 1, heads, d).contiguous()
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    parent = torch.full((rows, nodes), -1, dtype=torch.int32, device="cuda")
    got = wa.tree_decode(q, k, v, kt, -b, pos, parent, 0).double()
    l = 1.0 + p[..., None]
    want = (a.double() - p[..., None] * b.double()) / l
    assert want.abs().max() < 2 ** -6
    tol = (b.double() * (2 ** -18 + 2 ** -21) + 2 ** -21) / l + want.abs() * (2 ** -8 + 2 ** -17)
    off = (got - want).abs() / tol
    assert off.max() <= 1.0, (off.max().item(), (off > 1).double().mean().item())


def test_windows_and_scales_of_other_types(wa):
    """A window or a scale that is no plain number of its kind is taken for what it is or refused by its name."""
    c = _case(2, 5, 4, 2, 128, 64, 90, [200, 30], seed=14)
    want = _run(wa, c)
    args = [c[x] for x in ("q", "k", "v", "k_tree", "v_tree", "pos", "parent")]
    ws = torch.empty(wa.tree_decode_ws_bytes(2, 5, 4, 2, 128, 64, 90), dtype=torch.uint8, device="cuda")
    for _ in range(20):       # an error left behind shows at once or once the interpreter has specialised the call
        for win in (64.0, np.int64(64), np.float32(64.0)):
            assert _eq(wa.tree_decode(*args, win), want)
            assert _eq(wa.tree_decode(*args, win, ws=ws, scale=np.float64(1.0)), want)
        for win in (None, "64", [64]):
            with pytest.raises(TypeError, match="win"):
                wa.tree_decode(*args, win)
        for scale in (None, "x"):
            with pytest.raises(TypeError, match="scale"):
                wa.tree_decode(*args, 64, scale=scale)
        with pytest.raises(ValueError, match="win"):
            wa.tree_decode(*args, 64.5)
    assert _eq(_run(wa, c), want)


@pytest.mark.parametrize("win", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 32 + 64, 2 ** 70])
def test_windows_past_32_bits_are_refused(wa, win):
    """Not taken modulo 2^32."""
    c = _case(2, 5, 4, 2, 128, 64, 90, [80, 30], seed=14)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for kw in ({}, dict(ws=ws)):
        with pytest.raises(ValueError, match="win"):
            wa.tree_decode(*[c[x] for x in ("q", "k", "v", "k_tree", "v_tree", "pos", "parent")], win, **kw)
