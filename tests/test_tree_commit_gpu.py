"""Kept nodes into the rings on the GPU: every bit of every ring against a plain copy."""
from __future__ import annotations

import pytest
import torch

from _util import bits, ensure_built
from oracle import tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def rnd(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def both(wa, kt, vt, kr, vr, path, length, pos):
    want = [[tree.commit(bits(t), bits(r), path, length, pos) for t, r in zip(ts, rs)] for ts, rs in ((kt, kr), (vt, vr))]
    ws = wa.tree_commit(kt, vt, kr, vr, i32(path), i32(length), i32(pos))
    for rs, ws_ in zip((kr, vr), want):
        for r, w in zip(rs, ws_):
            assert (bits(r) == w).all()
    return wa.status(ws)


@pytest.mark.parametrize("rows,nodes,hkv,d,rings,length,pos", [
    (1, 1, 1, 128, [1], [1], [-1]),
    (1, 8, 8, 256, [1536], [4], [1534]),                       # wraps
    (3, 16, 2, 128, [50, 17, 1111], [16, 0, 7], [48, 3, 2 ** 31 - 20]),
    (2, 128, 1, 256, [200], [128, 100], [5, 199]),
    (5, 12, 16, 128, [64] * 64, [1, 2, 3, 4, 5], [0, 10, 62, 63, 64]),
    (2, 20, 3, 128, [6, 13], [20, 9], [4, 100]),               # more nodes than slots: the last ones stay
])
def test_copies(wa, rows, nodes, hkv, d, rings, length, pos):
    L = len(rings)
    kt, vt = [[rnd(rows, nodes, hkv, d) for _ in range(L)] for _ in range(2)]
    kr, vr = [[rnd(rows, x, hkv, d) for x in rings] for _ in range(2)]
    path = [sorted(torch.randperm(nodes)[:length[r]].tolist()) + [-1] * (nodes - length[r]) for r in range(rows)]
    assert both(wa, kt, vt, kr, vr, path, length, pos) == 0


def test_one_layer_without_lists_and_strided_nodes(wa):
    """A single layer's tensors as they are; v as a view of a projection buffer, k with nodes before rows."""
    rows, nodes, hkv, d = 3, 6, 2, 128
    fused = rnd(rows, nodes, 8 * d)
    vt = fused[:, :, 6 * d:].unflatten(2, (hkv, d))
    kt = rnd(nodes, rows, hkv, d).transpose(0, 1)
    kr, vr = rnd(rows, 9, hkv, d), rnd(rows, 9, hkv, d)
    path, length, pos = [[0, 2, 5], [1, 1, 1], [4, -1, -1]], [3, 2, 1], [7, 8, -1]
    want = [tree.commit(bits(t), bits(r), path, length, pos) for t, r in ((kt, kr), (vt, vr))]
    wa.tree_commit(kt, vt, kr, vr, i32(path), i32(length), i32(pos))
    assert (bits(kr) == want[0]).all() and (bits(vr) == want[1]).all()


def test_status(wa):
    rows, nodes = 3, 5
    mk = lambda m: [rnd(rows, m, 2, 128)]     # noqa: E731
    a = dict(kt=mk(nodes), vt=mk(nodes), kr=mk(11), vr=mk(11))
    ok = [[0, 1, 2], [0, 1, 2], [0, 1, 2]]
    assert both(wa, **a, path=ok, length=[3, 3, 3], pos=[0, 1, 2]) == 0
    assert both(wa, **a, path=ok, length=[3, 3, 3], pos=[0, -2, 2]) == wa.WA_STATUS_BAD_POS
    assert both(wa, **a, path=ok, length=[3, 4, 3], pos=[0, 1, 2]) == wa.WA_STATUS_BAD_TREE
    assert both(wa, **a, path=ok, length=[3, -1, 3], pos=[0, 1, 2]) == wa.WA_STATUS_BAD_TREE
    for bad in (5, -1, 2 ** 31 - 1, -2 ** 31):
        path = [[0, 1, 2], [0, bad, 2], [0, 1, 2]]
        assert both(wa, **a, path=path, length=[3, 3, 3], pos=[0, 1, 2]) == wa.WA_STATUS_BAD_TREE
    assert both(wa, **a, path=[[0, 1, 9], [0, 1, 2], [0, 1, 2]], length=[2, 3, 3], pos=[0, 1, 2]) == 0


def test_refusals(wa):
    t, r, p = rnd(2, 4, 2, 128), rnd(2, 9, 2, 128), i32([[0], [0]])
    one = i32([1, 1])
    with pytest.raises(ValueError):
        wa.tree_commit([t], [t], [r], [r, r], p, one, one)
    with pytest.raises(ValueError):
        wa.tree_commit([], [], [], [], p, one, one)
    with pytest.raises(ValueError):
        wa.tree_commit(t, t, r, rnd(2, 8, 2, 128)[:, :, :1], p, one, one)
    with pytest.raises(ValueError):
        wa.tree_commit([t, t], [t, rnd(2, 4, 3, 128)], [r, r], [r, r], p, one, one)
    with pytest.raises(ValueError):
        wa.tree_commit(t, t, r, r, p, i32([1]), one)
    with pytest.raises(ValueError):
        wa.tree_commit(t, t, r, r, one, one, one)


def test_in_a_graph(wa):
    kt, vt = rnd(2, 6, 4, 256), rnd(2, 6, 4, 256)
    kr, vr = rnd(2, 20, 4, 256), rnd(2, 20, 4, 256)
    path, length, pos = i32([[0, 1, 3], [0, 2, -1]]), i32([3, 2]), i32([18, 4])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    before = [kr.clone(), vr.clone()]
    wa.tree_commit(kt, vt, kr, vr, path, length, pos, ws=ws)
    kr.copy_(before[0])
    vr.copy_(before[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wa.tree_commit(kt, vt, kr, vr, path, length, pos, ws=ws, stream=s)
        pos.add_(length)
    k, v, at = bits(kr), bits(vr), pos.tolist()
    for _ in range(4):
        kt.neg_()
        k, v = tree.commit(bits(kt), k, path.tolist(), [3, 2], at), tree.commit(bits(vt), v, path.tolist(), [3, 2], at)
        at = [at[0] + 3, at[1] + 2]
        g.replay()
        torch.cuda.synchronize()
        assert (bits(kr) == k).all() and (bits(vr) == v).all() and pos.tolist() == at and wa.status(ws) == 0


def test_many_rows_report_their_own_faults(wa):
    """More entries than the one block looks through: the status is cleared and gathered instead."""
    rows, nodes, most = 700, 64, 64
    kt, vt, kr, vr = (rnd(rows, m, 1, 128) for m in (nodes, nodes, 80, 80))
    gen = torch.Generator().manual_seed(3)
    path = torch.randint(0, nodes, (rows, most), generator=gen).tolist()
    length = torch.randint(0, most + 1, (rows,), generator=gen).tolist()
    pos = torch.randint(-1, 10 ** 6, (rows,), generator=gen).tolist()
    args = dict(kt=[kt], vt=[vt], kr=[kr], vr=[vr])
    assert both(wa, **args, path=path, length=length, pos=pos) == 0
    length[-1] = 5
    path[-1][3] = nodes
    assert both(wa, **args, path=path, length=length, pos=pos) == wa.WA_STATUS_BAD_TREE
    path[-1][3], pos[0] = 0, -9
    assert both(wa, **args, path=path, length=length, pos=pos) == wa.WA_STATUS_BAD_POS
    pos[0], length[350] = 0, most + 1
    assert both(wa, **args, path=path, length=length, pos=pos) == wa.WA_STATUS_BAD_TREE


def test_one_ring_that_layers_share(wa):
    """A cache of two layers, and keys that are the values: the same tree into the same ring; other trees are refused."""
    t, other, r = rnd(2, 6, 2, 128), rnd(2, 6, 2, 128), rnd(2, 9, 2, 128)
    path, length, pos = [[0, 2, 5], [1, 3, -1]], [3, 2], [7, 3]
    want = tree.commit(bits(t), bits(r), path, length, pos)
    wa.tree_commit([t, t], [t, t], [r, r], [r, r], i32(path), i32(length), i32(pos))
    assert (bits(r) == want).all()
    for kt, vt in (([t, other], [t, t]), ([t, t], [other, other])):
        with pytest.raises(wa.WAError):
            wa.tree_commit(kt, vt, [r, r], [r, r], i32(path), i32(length), i32(pos))
    assert (bits(r) == want).all()
