"""Float64 definitions of the calls for drafted tokens: tree decode, verification, commit (TEST INFRASTRUCTURE).

Plain loops over rows, nodes and children, sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from . import attend, bf16_to_f64


def parent_of(parents, i: int) -> int:
    """Node i's parent; a value outside [-1, i) counts as -1."""
    p = int(parents[i])
    return p if -1 <= p < i else -1


def chain(parents, i: int) -> list:
    """Node i, its parent, its parent's parent, ... up to the root."""
    out = [i]
    while (i := parent_of(parents, i)) >= 0:
        out.append(i)
    return out


def decode(q, k, v, kt, vt, pos, parent, win: int, scale: float, n=None) -> np.ndarray:
    """Tree decode.  q [R,T,hq,d], k/v [R,ring,hkv,d], kt/vt [R,T,hkv,d] bf16 bits, pos [R], parent [R,T].

    Returns float64 [R,T,hq,d]; nodes past n are left NaN."""
    R, T, hq, d = q.shape
    ring, hkv = k.shape[1], k.shape[2]
    G = hq // hkv
    out = np.full((R, T, hq, d), np.nan)
    for r in range(R):
        p = max(int(pos[r]), -1)
        p = min(p, ring - 1) if win == 0 else p
        for i in range(T if n is None else min(max(int(n[r]), 0), T)):
            up = chain(parent[r], i)
            at = p + len(up)                                   # the node's own position
            lo = max(0, at - win + 1) if win > 0 else 0
            slots = np.arange(lo, p + 1, dtype=np.int64) % ring
            near = [a for back, a in enumerate(up) if win == 0 or back < win]
            for g in range(hkv):
                kk = np.concatenate([bf16_to_f64(k[r, slots, g]), bf16_to_f64(kt[r, near, g])])
                vv = np.concatenate([bf16_to_f64(v[r, slots, g]), bf16_to_f64(vt[r, near, g])])
                hs = slice(g * G, g * G + G)
                out[r, i, hs] = attend(bf16_to_f64(q[r, i, hs]), kk, vv, scale)[0]
    return out


def prob(x) -> np.ndarray:
    """Probabilities as the verification takes them: NaN and negative values are 0, those above 1 are 1."""
    x = np.asarray(x, dtype=np.float64)
    return np.where(x > 0, np.minimum(x, 1.0), 0.0)


def verify(target, draft, parent, tokens, u, n=None):
    """Verification: target / draft [R,T,V] (draft may be None), parent / tokens [R,T], u [R,T].

    Returns (path [R,T], length [R], token [R]) as lists."""
    R, T, V = np.shape(target)
    paths, lengths, out = [], [], []
    for r in range(R):
        nr = T if n is None else min(max(int(n[r]), 0), T)
        if nr == 0:
            paths.append([-1] * T)
            lengths.append(0)
            out.append(-1)
            continue
        path = [0]
        while True:
            node = path[-1]
            w, s = prob(target[r][node]), 1.0
            q = None if draft is None else prob(draft[r][node])
            kept = False
            for c in range(node + 1, nr):
                x = int(tokens[r][c])
                if parent_of(parent[r], c) != node or not 0 <= x < V:
                    continue
                qx = 1.0 if q is None else q[x]
                if float(u[r][c]) * qx * s < w[x]:
                    path.append(c)
                    kept = True
                    break
                if q is None:
                    left = w.copy()
                    left[x] = 0.0
                else:
                    left = np.maximum(w - s * q, 0.0)
                if left.sum() > 0:
                    w, s = left, left.sum()
            if not kept:
                break
        run = np.cumsum(w)
        hit = np.nonzero((run > float(u[r][0]) * run[-1]) & (w > 0))[0]
        some = np.nonzero(w > 0)[0]
        out.append(int(hit[0]) if hit.size else int(some[-1]) if some.size else -1)
        paths.append(path + [-1] * (T - len(path)))
        lengths.append(len(path))
    return paths, lengths, out


def commit(tree, ring, path, length, pos):
    """Kept nodes into a ring: tree [R,T,...], ring [R,ring,...] (any dtype); returns the new ring."""
    ring = ring.copy()
    R, T = tree.shape[:2]
    most = np.shape(path)[1]
    for r in range(R):
        if pos[r] < -1:
            continue
        for j in range(min(max(int(length[r]), 0), most)):
            if 0 <= path[r][j] < T:
                ring[r, (int(pos[r]) + 1 + j) % ring.shape[1]] = tree[r, path[r][j]]
    return ring
