"""The calls for drafted tokens as a serving loop runs them: preparation, attention, verification, commit.

Two layers (a sliding one and a linear one) and three sequences take several drafted steps.  After each, every kept
node is decoded again one token at a time through `decode` from the rings that the commit filled: both calls have to
lie in the decode form's range around the float64 value, which is computed from the rings alone.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import wa_synth
from _util import assert_parity, bits, ensure_built
from oracle import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("kind", ["chain", "bushy"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 256), (6, 2, 128)])
def test_drafted_steps(wa, kind, hq, hkv, d):
    rows, nodes, V = 3, 10, 500
    gen = torch.Generator(device="cuda").manual_seed(3)
    layers = [(48, 60), (0, 200)]                                 # (win, ring)
    pos = torch.tensor([70, 59, -1], dtype=torch.int32, device="cuda")
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)   # noqa: E731
    kr, vr = [[rnd(rows, ring, hkv, d) * (0.1 if x == 0 else 1) for _, ring in layers] for x in range(2)]
    inv = torch.from_numpy((1.0 / 10000.0 ** (np.arange(0, d, 2) / d)).astype(np.float32)).cuda()
    parents = wa_synth.draft_tree(kind, nodes, 1)
    depth = [0] * nodes
    for i in range(1, nodes):
        depth[i] = depth[parents[i]] + 1
    parent = torch.tensor([parents] * rows, dtype=torch.int32, device="cuda")
    depth = torch.tensor(depth, dtype=torch.int32, device="cuda")
    scale = 4.0
    kept_several = 0
    for step in range(3):
        node_pos = (pos[:, None] + 1 + depth).flatten().contiguous()
        qs, kt, vt, outs = [], [], [], []
        for layer, (win, _) in enumerate(layers):
            src = rnd(rows * nodes, (hq + 2 * hkv) * d)
            q = torch.empty((rows * nodes, hq, d), dtype=torch.bfloat16, device="cuda")
            k = torch.empty((rows * nodes, 1, hkv, d), dtype=torch.bfloat16, device="cuda")
            wa.prep_append(src, node_pos, q, k, None, mode="l2_rope", inv_freq=inv)
            qs.append(q.view(rows, nodes, hq, d))
            kt.append(k.view(rows, nodes, hkv, d))
            # v stays where the projection left it
            vt.append(src.view(rows, nodes, -1)[:, :, (hq + hkv) * d:].unflatten(2, (hkv, d)))
            outs.append(wa.tree_decode(qs[-1], kr[layer], vr[layer], kt[-1], vt[-1], pos, parent, win, scale=scale))
        logits = torch.randn((rows, nodes, V), generator=gen, device="cuda") * 2
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits + 0.5 * torch.randn((rows, nodes, V), generator=gen, device="cuda"), -1)
        at = parent.long().clamp_min(0)
        drawn = torch.multinomial(draft[torch.arange(rows, device="cuda")[:, None], at].view(-1, V), 1, generator=gen)
        path, length, token = wa.tree_verify(target, parent, drawn.view(rows, nodes).int(),
                                             torch.rand((rows, nodes), generator=gen, device="cuda"), draft=draft)
        ws = wa.tree_commit(kt, vt, kr, vr, path, length, pos)
        assert wa.status(ws) == 0
        assert (length >= 1).all() and (token >= 0).all()
        kept_several += int((length > 1).sum())

        for layer, (win, ring) in enumerate(layers):
            k, v = bits(kr[layer]), bits(vr[layer])
            for j in range(int(length.max())):
                # the rows that kept a j-th node, decoded at its position; the window of a ring without spare slots
                # reaches back at most ring - (nodes kept after it) keys
                who = [r for r in range(rows) if int(length[r]) > j and (win == 0 or win + int(length[r]) - j <= ring + 1)]
                node = [int(path[r, j]) for r in who]
                p = [int(pos[r]) + 1 + j for r in who]
                q1 = qs[layer][who, node].contiguous()
                one = wa.decode(q1, kr[layer][who].contiguous(), vr[layer][who].contiguous(),
                                torch.tensor(p, dtype=torch.int32, device="cuda"), win, scale)
                ref = oracle.decode(bits(q1), k[who], v[who], p, win, ring, scale)
                assert_parity(one, ref, check.TOL_FP32_P, "decode")
                assert_parity(outs[layer][who, node], ref, check.TOL_FP32_P, "tree decode")
        pos = pos + length
    assert kept_several > 0
