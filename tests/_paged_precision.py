"""Paged-decode inputs whose outputs show what a kernel's P and its queries lose, with bounds worked out beside them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged

LIVE = 8          # keys with a weight worth mentioning, all in one tile
FAR = -64.0       # the score of every other key: a weight of 2^-92


def weights(t, parts, bits):
    """exp(t), largest 1, as `parts` bf16 or e4m3 numbers hold them: the first of the weight (8 bits: of 256 times it),
    each next of what is left (8 bits: 32 times that)."""
    w = np.exp(np.asarray(t, dtype=np.float64)) * (256.0 if bits == 8 else 1.0)
    rest, total, unit = w.copy(), np.zeros_like(w), 1.0
    for _ in range(parts):
        if bits == 8:
            e = paged.e4m3_to_f64(paged.f64_to_e4m3(rest))
        else:
            e = torch.from_numpy(rest).float().to(torch.bfloat16).double().numpy()
        total += e * unit
        rest = rest - e
        if bits == 8:
            rest, unit = rest * 32, unit / 32
    return total / (256.0 if bits == 8 else 1.0)


def cancelling(d, seed):
    """(t [LIVE], v [LIVE, d]) of whole e4m3 numbers: weights exp(t) between 1/e and 1 whose values nearly cancel in every dim, so
    that a weight's error of 2^-k shows as one of about 2^-k in an output of less than 2^-11, whose own rounding is below 2^-19."""
    rng = np.random.default_rng(seed)
    grid = np.arange(8, 17) / 16.0
    t = -np.concatenate([[0.0], rng.choice(np.concatenate([grid, grid[:-1] / 2]), LIVE - 1, replace=False)])
    w = np.exp(t)
    some = np.concatenate([s * (8 + np.arange(8)) / 8.0 * 2.0 ** e for s in (-1, 1) for e in (-1, 0)])
    v = np.zeros((LIVE, d))
    i = np.stack(np.meshgrid(some, some, some, indexing="ij"), -1).reshape(-1, 3)
    sums = i @ w[LIVE - 3:]
    order = np.argsort(sums)
    sums, i = sums[order], i[order]
    todo = np.arange(d)
    while len(todo):                  # all but three at random, those so that the sum is next to zero
        v[:LIVE - 3, todo] = rng.choice(some, (LIVE - 3, len(todo)))
        at = np.clip(np.searchsorted(sums, -(w[:LIVE - 3] @ v[:LIVE - 3, todo])), 0, len(sums) - 1)
        v[LIVE - 3:, todo] = i[at].T
        todo = todo[np.abs(w @ v[:, todo]) > 2.0 ** -12 * w.sum()]
    return t, v


def place(c, rows, t, v):
    """Puts the scores t[r] and the values v[r] at the positions rows[r] of a case of wa_synth.paged_case whose keys have scores
    along dim 0 of a query that is 1 there and 0 elsewhere."""
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    for x in "kv":
        c[x].copy_(torch.zeros((), device=c[x].device))
    c["k"][..., 0] = torch.full((), FAR, device=c["k"].device).to(c["k"].dtype)
    c["k_scale"] = c["v_scale"] = None
    page = c["k"].shape[1]
    for r, at in enumerate(rows):
        for j, p in enumerate(at):
            i = int(c["table"][r, p // page])
            c["k"][i, p % page, :, 0] = torch.full((), float(t[r][j]), device=c["k"].device).to(c["k"].dtype)
            c["v"][i, p % page] = torch.from_numpy(v[r][j]).to(c["v"].device).float().to(c["v"].dtype)
