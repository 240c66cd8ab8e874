"""The float64 definitions for drafted tokens, pinned on small cases (CPU).

The tree decode's against the decode definition (a node is a decode row on a cache that holds its ancestors),
the verification's against exact fractions and against what it promises (the kept tokens and the sampled one
are distributed as the target's own), the commit's against a hand-made ring.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import wa_synth
from oracle import tree


def _bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("win,ring,pos", [(0, 40, 20), (7, 9, 30), (3, 40, 12), (1, 5, 4), (7, 9, -1), (0, 40, -1)])
@pytest.mark.parametrize("kind", ["chain", "random", "flat"])
def test_a_node_is_a_decode_row_on_a_cache_that_holds_its_ancestors(win, ring, pos, kind):
    T = 8
    c = wa_synth.tree_case(1, T, 2, 1, 128, win, ring, [pos], seed=3, kind=kind)
    k, v, kt, vt = (_bits(c[x]) for x in ("k", "v", "k_tree", "v_tree"))
    parent = c["parent"].numpy()
    got = tree.decode(_bits(c["q"]), k, v, kt, vt, [pos], parent, win, 1.0)
    for i in range(T):
        up = tree.chain(parent[0], i)[::-1]
        # a linear cache long enough for the row and its drafts
        full = pos + 1 + len(up)
        k2 = np.zeros((1, full, 1, 128), dtype=np.uint16)
        v2 = np.zeros_like(k2)
        for j in range(max(0, pos + 1 - ring), pos + 1):
            k2[0, j], v2[0, j] = k[0, j % ring], v[0, j % ring]
        for j, a in enumerate(up):
            k2[0, pos + 1 + j], v2[0, pos + 1 + j] = kt[0, a], vt[0, a]
        want = oracle.decode(_bits(c["q"])[:, i], k2, v2, [full - 1], win, full, 1.0)
        np.testing.assert_allclose(got[0, i], want[0], rtol=1e-12, atol=1e-12)


def _verify_fractions(p, q, children, tokens, u):
    """One node with leaves below it: (kept child or None, token), in exact fractions."""
    w, s = [Fraction(float(x)) for x in p], Fraction(1)
    for c in children:
        x = tokens[c]
        qx = Fraction(1) if q is None else Fraction(float(q[x]))
        if Fraction(float(u[c])) * qx * s < w[x]:
            return c
        left = [Fraction(0) if i == x else y for i, y in enumerate(w)] if q is None else \
            [max(y - s * Fraction(float(z)), Fraction(0)) for y, z in zip(w, q)]
        if sum(left) > 0:
            w, s = left, sum(left)
    run, total = Fraction(0), sum(w)
    for x, y in enumerate(w):
        run += y
        if run > Fraction(float(u[0])) * total:
            return ("token", x)


@pytest.mark.parametrize("with_draft", [True, False])
def test_verification_follows_its_definition_in_fractions(with_draft):
    rng = np.random.default_rng(5)
    for _ in range(200):
        V, kids = 7, int(rng.integers(1, 5))
        T = kids + 1
        p, q = rng.dirichlet(np.full(V, 0.6), 2).astype(np.float32)
        target = np.tile(p, (1, T, 1))
        draft = np.tile(q, (1, T, 1)) if with_draft else None
        tokens = np.concatenate([[0], rng.choice(V, kids, p=q.astype(np.float64) / q.astype(np.float64).sum())])
        u = rng.random((1, T)).astype(np.float32)
        path, length, token = tree.verify(target, draft, [[-1] + [0] * kids], [tokens], u)
        want = _verify_fractions(p, q if with_draft else None, range(1, T), tokens, u[0])
        if isinstance(want, tuple):
            assert length == [1] and token == [want[1]]
        else:
            assert length == [2] and path[0][:2] == [0, want]


@pytest.mark.parametrize("kids", [1, 3])
def test_the_first_token_after_the_root_is_distributed_as_the_target(kids):
    """Children drawn from q, verified against p: the token that follows node 0 (a kept child's, or the sampled
    one) has the target's distribution.  30,000 walks: a share's standard deviation is at most 0.0029, and the
    six shares are held to four of them."""
    rng = np.random.default_rng(11)
    V, walks = 6, 30000
    p = np.array([0.4, 0.05, 0.25, 0.1, 0.2, 0.0], dtype=np.float32)
    q = np.array([0.1, 0.3, 0.25, 0.05, 0.1, 0.2], dtype=np.float32)
    T = kids + 1
    tokens = rng.choice(V, (walks, T), p=q.astype(np.float64) / q.astype(np.float64).sum())
    u = rng.random((walks, T)).astype(np.float32)
    target, draft = np.broadcast_to(p, (walks, T, V)), np.broadcast_to(q, (walks, T, V))
    path, length, token = tree.verify(target, draft, np.tile([-1] + [0] * kids, (walks, 1)), tokens, u)
    after = [tokens[i, path[i][1]] if length[i] > 1 else token[i] for i in range(walks)]
    share = np.bincount(after, minlength=V) / walks
    assert np.all(np.abs(share - p) < 4 * np.sqrt(0.25 / walks)), share
    assert share[5] == 0


def test_verification_of_degenerate_rows():
    V = 4
    p = np.array([[0.5, 0.5, 0, 0]], dtype=np.float32)
    one = lambda x: np.array([[x]], dtype=np.float32)   # noqa: E731
    # thresholds on a border take the next token; past the end, the last one with weight
    assert tree.verify(p[None], None, [[-1]], [[0]], one(0.0))[2] == [0]
    assert tree.verify(p[None], None, [[-1]], [[0]], one(0.5))[2] == [1]
    assert tree.verify(p[None], None, [[-1]], [[0]], one(1.0))[2] == [1]
    assert tree.verify(p[None], None, [[-1]], [[0]], one(np.nan))[2] == [1]
    # no mass, no nodes, NaN and negative probabilities
    assert tree.verify(np.zeros((1, 1, V)), None, [[-1]], [[0]], one(0.3)) == ([[0]], [1], [-1])
    assert tree.verify(p[None], None, [[-1]], [[0]], one(0.3), n=[0]) == ([[-1]], [0], [-1])
    assert tree.verify(np.array([[[np.nan, -1, 0.25, 0]]]), None, [[-1]], [[0]], one(0.3))[2] == [2]


def test_commit_wraps_and_skips():
    tr = np.arange(2 * 5 * 1).reshape(2, 5, 1) + 100
    ring = np.zeros((2, 4, 1), dtype=tr.dtype)
    got = tree.commit(tr, ring, [[0, 2, 4, -1], [1, 9, 3, -1]], [3, 4], [6, -1])
    assert got[0, :, 0].tolist() == [102, 104, 0, 100]      # slots 3, 0, 1
    assert got[1, :, 0].tolist() == [106, 0, 108, 0]        # entry 9 is not a node
