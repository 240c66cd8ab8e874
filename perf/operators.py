"""Cases of the drafted-tree operators: attention of a tree of drafted tokens over a ring cache, the
verification of the drafts against the target's probabilities, and the move of the accepted nodes' keys and
values into the ring.

A step of a serving loop that drafts tokens runs the three in this order: per layer `tree_decode`, then
`tree_verify` on the target's probabilities, then `tree_commit`.  Node 0 of a row's tree is the last token
that was sampled (not in the cache yet), the others are drafts; parent[i] < i, -1 for a root.  `pos` is the
last position in the cache; node i stands at position pos + 1 + depth(i).

`run` computes each operator in its plain form, or with `own` set makes the package's calls.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one chat stream, a short draft over a sliding layer: a latency-bound call of every layer
        dict(name="decode_one_sliding", op="decode", rows=1, nodes=8, hq=16, hkv=8, d=256, win=1024, ring=1536,
             pos_lo=5000, pos_hi=5000, ragged=False, tree="chain"),
        # a full serving batch on a sliding layer: wrapped rings, positions of every age
        dict(name="decode_batch_sliding", op="decode", rows=64, nodes=16, hq=32, hkv=16, d=256, win=1024, ring=1536,
             pos_lo=100, pos_hi=40000, ragged=False, tree="random"),
        # one stream on a long linear cache: the key axis has to be split over the card
        dict(name="decode_one_linear", op="decode", rows=1, nodes=12, hq=16, hkv=8, d=256, win=0, ring=32768,
             pos_lo=32000, pos_hi=32000, ragged=False, tree="random"),
        # a batch on long linear caches, the largest read
        dict(name="decode_batch_linear", op="decode", rows=8, nodes=32, hq=32, hkv=16, d=256, win=0, ring=32768,
             pos_lo=9000, pos_hi=32700, ragged=False, tree="bushy"),
        # wide trees over groups of eight query heads: 512 query rows a key head, arithmetic counts
        dict(name="decode_wide_group8", op="decode", rows=32, nodes=64, hq=32, hkv=4, d=128, win=0, ring=16384,
             pos_lo=4000, pos_hi=16300, ragged=False, tree="bushy"),
        # ragged batch: groups of three heads, an odd ring, some rows without a draft, one empty cache
        dict(name="decode_ragged", op="decode", rows=13, nodes=27, hq=24, hkv=8, d=128, win=1000, ring=1111,
             pos_lo=-1, pos_hi=7000, ragged=True, tree="random"),
        # verification of one stream's short chain: latency
        dict(name="verify_one", op="verify", rows=1, nodes=8, vocab=32768, draft=True, ragged=False, tree="chain"),
        # verification of a batch of trees with the draft's probabilities
        dict(name="verify_batch", op="verify", rows=64, nodes=16, vocab=131072, draft=True, ragged=False,
             tree="random"),
        # trees of the draft's best tokens (no draft probabilities), an odd vocabulary, ragged rows
        dict(name="verify_points", op="verify", rows=24, nodes=26, vocab=100003, draft=False, ragged=True,
             tree="bushy"),
        # accepted nodes of one stream into one layer's ring
        dict(name="commit_one", op="commit", layers=1, rows=1, nodes=8, hkv=8, d=256, ring=1536, take=4),
        # accepted nodes of a batch into the rings of a stack of layers
        dict(name="commit_stack", op="commit", layers=12, rows=48, nodes=16, hkv=8, d=256, ring=1536, take=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "verify", "verify", "commit"])
    if op == "decode":
        d = rng.choice([128, 256])
        hkv = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        if hkv * group > 64:
            group = 2
        win = rng.choice([0, 0, _log(rng, 100, 4096)])
        span = win if win else _log(rng, 300, 32768)
        nodes = _log(rng, 1, 128)
        rows = _log(rng, 1, 64)
        # at most the products of the largest listed case, and 2 GB of keys and values
        while rows > 1 and (rows * nodes * hkv * group * span * d > 8e10 or rows * span * hkv * d * 4 > 2e9):
            rows = max(1, rows // 2)
        while nodes > 1 and rows * nodes * hkv * group * span * d > 8e10:
            nodes = max(1, nodes // 2)
        ring = span + (rng.randint(0, 700) if win else rng.randint(1, 64))
        lo = rng.choice([-1, span // 4, span // 2])
        hi = rng.randint(lo + 1, 60000) if win else ring - 1
        return dict(op="decode", rows=rows, nodes=nodes, hq=hkv * group, hkv=hkv, d=d, win=win, ring=ring,
                    pos_lo=lo, pos_hi=hi, ragged=rng.random() < 0.5, tree=rng.choice(["chain", "random", "bushy"]))
    if op == "verify":
        vocab = _log(rng, 1000, 140000)
        nodes = _log(rng, 1, 64)
        rows = _log(rng, 1, 64)
        while rows > 1 and rows * nodes * vocab > 64 * 16 * 131072:
            rows = max(1, rows // 2)
        return dict(op="verify", rows=rows, nodes=nodes, vocab=vocab, draft=rng.random() < 0.6,
                    ragged=rng.random() < 0.5, tree=rng.choice(["chain", "random", "bushy"]))
    rows, layers = _log(rng, 1, 48), _log(rng, 1, 12)
    hkv, d, nodes = rng.choice([1, 2, 4, 8]), rng.choice([128, 256]), _log(rng, 2, 64)
    return dict(op="commit", layers=layers, rows=rows, nodes=nodes, hkv=hkv, d=d, ring=rng.randint(200, 1536),
                take=rng.randint(1, nodes))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, rows):
    """`rows` whole numbers from lo to hi, evenly apart."""
    return [lo + (hi - lo) * i // max(1, rows - 1) for i in range(rows)] if rows > 1 else [hi]


def _counts(case):
    """Nodes of each row: all of them, or spread from all to none."""
    rows, nodes = case["rows"], case["nodes"]
    return _spread(nodes, 0, rows) if case["ragged"] and rows > 1 else [nodes] * rows


def _parents(kind, nodes, r):
    """A tree over `nodes` nodes, parents before children, node 0 its root."""
    if kind == "chain":
        return [i - 1 for i in range(nodes)]
    if kind == "bushy":     # three children a node, level by level
        return [-1] + [(i - 1) // 3 for i in range(1, nodes)]
    return [-1] + [r.randint(max(0, i - 6), i - 1) for i in range(1, nodes)]


def _trees(case, r):
    parents = [_parents(case["tree"], case["nodes"], r) for _ in range(case["rows"])]
    depths, ranks = [], []
    for p in parents:
        dep, rank, kids = [], [], {}
        for i, a in enumerate(p):
            dep.append(0 if a < 0 else dep[a] + 1)
            rank.append(kids.get(a, 0))
            kids[a] = rank[-1] + 1
        depths.append(dep)
        ranks.append(rank)
    return parents, depths, ranks


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bf16(shape, gen, rms=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, rms, generator=gen)


def prepare(case, seed):
    r = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed * 1009 + 17)
    rows, nodes = case["rows"], case["nodes"]
    s = dict(case)
    if case["op"] == "decode":
        hq, hkv, d, ring = case["hq"], case["hkv"], case["d"], case["ring"]
        order = list(range(rows))
        r.shuffle(order)
        pos = _spread(case["pos_lo"], case["pos_hi"], rows)
        n = _counts(case)
        parents, depths, _ = _trees(case, r)
        s["q"] = _bf16((rows, nodes, hq, d), gen)
        # keys of RMS 0.1 at scale 1 for head dim 256, unit keys at scale 1 / sqrt(d) for 128
        krms, s["scale"] = (0.1, 1.0) if d == 256 else (1.0, 1.0 / math.sqrt(d))
        s["k_ring"], s["v_ring"] = _bf16((rows, ring, hkv, d), gen, krms), _bf16((rows, ring, hkv, d), gen)
        s["k_tree"], s["v_tree"] = _bf16((rows, nodes, hkv, d), gen, krms), _bf16((rows, nodes, hkv, d), gen)
        s["pos"], s["n"] = _i32([pos[i] for i in order]), _i32([n[i] for i in order])
        s["parent"], s["depth"] = _i32(parents), _i32(depths)
        # peaked keys: the i-th key from the end lies along a query of node i, in each key head, at a score of
        # about 10, so that some rows lean on one key and the others on all of them
        rise, heads = (0.04 if d == 256 else 0.9), torch.arange(hkv, device="cuda") * (hq // hkv)
        row = torch.arange(rows, device="cuda")
        for i in range(min(nodes, ring)):
            s["k_ring"][row, (s["pos"].long() - i) % ring] = s["q"][:, i, heads + i % (hq // hkv)] * rise
        s["out"] = torch.zeros((rows, nodes, hq, d), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "verify":
        V = case["vocab"]
        parents, depths, ranks = _trees(case, r)
        n = _counts(case)
        r.shuffle(n)
        logits = torch.empty((rows, nodes, V), device="cuda").normal_(0.0, 3.0, generator=gen)
        s["target"] = torch.softmax(logits, -1)
        # the draft model's logits are the target's with noise, which accepts most first drafts
        draft = torch.softmax(logits.add_(torch.randn((rows, nodes, V), generator=gen, device="cuda")), -1)
        s["parent"], s["n"] = _i32(parents), _i32(n)
        s["steps"], s["branch"] = max(map(max, depths)), 1 + max(map(max, ranks))
        at = s["parent"].long().clamp_min(0)
        rank = _i32(ranks).long()
        if case["draft"]:    # a node's children are drawn from the draft's distribution there
            every = torch.multinomial(draft.view(rows * nodes, V), s["branch"], replacement=True, generator=gen)
            s["draft"] = draft
        else:                # a node's children are the draft's best tokens there
            every, s["draft"] = torch.topk(draft.view(rows * nodes, V), s["branch"]).indices, None
        every = every.view(rows, nodes, s["branch"])
        row = torch.arange(rows, device="cuda")[:, None]
        s["tokens"] = every[row, at, rank].int()
        s["u"] = torch.rand((rows, nodes), generator=gen, device="cuda")
    else:
        L, hkv, d, ring, take = case["layers"], case["hkv"], case["d"], case["ring"], case["take"]
        for name, size in (("k_tree", nodes), ("v_tree", nodes), ("k_ring", ring), ("v_ring", ring)):
            s[name] = [_bf16((rows, size, hkv, d), gen) for _ in range(L)]
        path = [sorted(r.sample(range(nodes), take)) + [-1] * (nodes - take) for _ in range(rows)]
        s["path"] = _i32(path)
        s["length"] = _i32([take] * rows)
        s["pos"] = _i32([r.randint(-1, 40000) for _ in range(rows)])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if s["op"] == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    if s["op"] == "verify":
        return _own_verify(s) if own else _plain_verify(s)
    return _own_commit(s) if own else _plain_commit(s)


def _own_decode(s):
    import sliding_window_gqa_gb300 as wa
    return wa.tree_decode(s["q"], s["k_ring"], s["v_ring"], s["k_tree"], s["v_tree"], s["pos"], s["parent"],
                          s["win"], n=s["n"], scale=s["scale"], out=s["out"])


def _own_verify(s):
    import sliding_window_gqa_gb300 as wa
    path, length, token = wa.tree_verify(s["target"], s["parent"], s["tokens"], s["u"], draft=s["draft"], n=s["n"])
    return {"path": path, "length": length, "token": token}


def _own_commit(s):
    import sliding_window_gqa_gb300 as wa
    wa.tree_commit(s["k_tree"], s["v_tree"], s["k_ring"], s["v_ring"], s["path"], s["length"], s["pos"])
    return {"k": s["k_ring"], "v": s["v_ring"]}


def _ancestors(parent, steps):
    """[rows, nodes, nodes] truth values: column j is an ancestor of node i, or i itself."""
    rows, nodes = parent.shape
    eye = torch.eye(nodes, dtype=torch.bool, device=parent.device).expand(rows, nodes, nodes)
    # reach doubles each time: reach = one step; (reach or itself) squared
    see = eye | (parent.long()[:, :, None] == torch.arange(nodes, device=parent.device))
    for _ in range(max(1, math.ceil(math.log2(max(2, steps))))):
        see = torch.matmul(see.float(), see.float()) > 0
    return see


def _plain_decode(s):
    rows, nodes, hq, d = s["q"].shape
    _, ring, hkv, _ = s["k_ring"].shape
    win, G, dev = s["win"], hq // hkv, s["q"].device
    span = min(ring, win) if win else ring
    pos, depth = s["pos"].long(), s["depth"].long()
    # the last `span` positions of every row, oldest first (a linear cache: all of its slots)
    at = torch.arange(span, device=dev)[None] + ((pos + 1)[:, None] - span if win else 0)
    slot = at.clamp_min(0) % ring
    row = torch.arange(rows, device=dev)[:, None]
    in_cache = (at >= 0) & (at <= pos[:, None])
    first = pos[:, None] + 1 + depth - win + 1 if win else torch.zeros_like(depth)
    see_ring = in_cache[:, None] & (at[:, None] >= first[:, :, None])
    see_tree = _ancestors(s["parent"], nodes)
    if win:
        see_tree = see_tree & (depth[:, :, None] - depth[:, None] < win)
    see = torch.cat([see_ring, see_tree], 2)                                     # [rows, nodes, keys]
    k = torch.cat([s["k_ring"][row, slot] if win else s["k_ring"], s["k_tree"]], 1).float()
    v = torch.cat([s["v_ring"][row, slot] if win else s["v_ring"], s["v_tree"]], 1).float()
    q = s["q"].float().view(rows, nodes, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(rows, hkv, nodes * G, d)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).view(rows, hkv, nodes, G, -1).mul_(s["scale"])
    sc.masked_fill_(~see[:, None, :, None], -math.inf)
    sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    total = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc.view(rows, hkv, nodes * G, -1), v.permute(0, 2, 1, 3)).view(rows, hkv, nodes, G, d) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(rows, nodes, hq, d).to(torch.bfloat16)
    drafted = torch.arange(nodes, device=dev)[None] < s["n"].long()[:, None]
    return torch.where(drafted[:, :, None, None], o, s["out"])


def _plain_verify(s):
    """The walk from node 0, all rows together: at most `branch` children of at most `steps` nodes."""
    p, q, parent, tokens, u = s["target"], s["draft"], s["parent"].long(), s["tokens"].long(), s["u"].double()
    rows, nodes, V = p.shape
    dev = p.device
    row = torch.arange(rows, device=dev)
    idx = torch.arange(nodes, device=dev)[None]
    n = s["n"].long()
    node = torch.zeros(rows, dtype=torch.long, device=dev)
    live = n > 0
    path = torch.full((rows, nodes), -1, dtype=torch.long, device=dev)
    path[:, 0] = torch.where(live, node, -1)
    length = live.long()
    weight = None
    for step in range(s["steps"] + 1):
        # the current node's weights: p, less the rejected drafts' share
        now = p[row, node].double()
        total, used, fresh = torch.ones(rows, dtype=torch.double, device=dev), 0.0, now
        took = torch.zeros_like(live)
        kids = (parent == node[:, None]) & (idx > node[:, None]) & (idx < n[:, None]) & live[:, None]
        for k in range(s["branch"] if step < s["steps"] else 0):
            kid = torch.where(kids.cumsum(1) == k + 1, kids, False)
            here = kid.any(1) & ~took
            child = kid.long().argmax(1)
            tok = tokens[row, child]
            share = torch.zeros_like(now).scatter_(1, tok[:, None], 1.0) if q is None else q[row, node].double()
            ok = here & (u[row, child] * share[row, tok] * total < fresh[row, tok])
            nxt = torch.where(share > 0, 0.0, fresh) if q is None else (fresh - total[:, None] * share).clamp_min(0.0)
            left = nxt.sum(1)
            drop = here & ~ok & (left > 0)
            fresh = torch.where(drop[:, None], nxt, fresh)
            total = torch.where(drop, left, total)
            path[row, length.clamp_max(nodes - 1)] = torch.where(ok, child, path[row, length.clamp_max(nodes - 1)])
            length = length + ok.long()
            go = child if k == 0 else torch.where(ok, child, go)
            took = took | ok
        stop = live & ~took
        weight = fresh if weight is None else torch.where(stop[:, None], fresh, weight)
        if step < s["steps"]:
            node = torch.where(took, go, node)
        live = live & took
    run_sum = weight.cumsum(1)
    mass = run_sum[:, -1:]
    token = (run_sum > u[:, :1] * mass).long().argmax(1)
    token = torch.where((n > 0) & (mass[:, 0] > 0), token, -1)
    return {"path": path.int(), "length": length.int(), "token": token.int()}


def _plain_commit(s):
    path, length, pos = s["path"].long(), s["length"].long(), s["pos"].long()
    rows, most = path.shape
    row = torch.arange(rows, device=path.device)[:, None]
    j = torch.arange(most, device=path.device)[None]
    take = (j < length[:, None])[:, :, None, None]
    at = path.clamp_min(0)
    for i in range(s["layers"]):
        slot = (pos[:, None] + 1 + j) % s["k_ring"][i].shape[1]
        for tree, ring in ((s["k_tree"][i], s["k_ring"][i]), (s["v_tree"][i], s["v_ring"][i])):
            ring[row, slot] = torch.where(take, tree[row, at], ring[row, slot])
    return {"k": s["k_ring"], "v": s["v_ring"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "decode":
        hq, hkv, d, win = case["hq"], case["hkv"], case["d"], case["win"]
        kv, dots, qo = 0, 0, 0
        for p, n in zip(_spread(case["pos_lo"], case["pos_hi"], case["rows"]), _counts(case)):
            if n:
                keys = min(p + 1, win - 1) if win else p + 1
                kv += keys + n
                dots += n * (keys + (n + 1) // 2)
                qo += n
        return {"bytes": 4 * kv * hkv * d + 4 * qo * hq * d, "flops": 4 * dots * hq * d}
    if case["op"] == "verify":
        live = sum(1 for n in _counts(case) if n)
        # the row of the node where each walk ends: its target, and its draft distribution where there is one
        return {"bytes": live * case["vocab"] * 4 * (2 if case["draft"] else 1), "flops": 4 * live * case["vocab"]}
    return {"bytes": 8 * case["layers"] * case["rows"] * case["take"] * case["hkv"] * case["d"], "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "commit":
        return None          # copies: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return _exact_verify(case, s)


def _exact_decode(case, s):
    """Row by row and key head by key head: the softmax over each node's visible keys."""
    rows, nodes, hq, hkv, d, win, ring = (case[x] for x in ("rows", "nodes", "hq", "hkv", "d", "win", "ring"))
    G = hq // hkv
    pos, n, parents = s["pos"].tolist(), s["n"].tolist(), s["parent"].tolist()
    out = torch.zeros((rows, nodes, hq, d), dtype=torch.float64, device="cuda")
    for r in range(rows):
        if n[r] == 0:
            continue
        lo = max(0, pos[r] + 2 - win) if win else 0
        at = torch.arange(lo, pos[r] + 1, device="cuda")
        kept = np.zeros((nodes, at.numel() + nodes), dtype=bool)
        for i in range(n[r]):
            chain, a = [], i
            while a >= 0:
                chain.append(a)
                a = parents[r][a]
            mine = pos[r] + len(chain)                       # the node's own position
            start = max(0, mine - win + 1) if win else 0
            kept[i, max(0, start - lo):at.numel()] = True
            for back, a in enumerate(chain):
                kept[i, at.numel() + a] = not win or back < win
        hide = torch.from_numpy(~kept).cuda()
        for g in range(hkv):
            keys = torch.cat([s["k_ring"][r, at % ring, g], s["k_tree"][r, :, g]]).double()
            vals = torch.cat([s["v_ring"][r, at % ring, g], s["v_tree"][r, :, g]]).double()
            for h in range(g * G, g * G + G):
                x = (s["q"][r, :, h].double() @ keys.T) * (1.0 if d == 256 else 1.0 / math.sqrt(d))
                x[hide] = -math.inf
                w = torch.softmax(x[:n[r]], -1)
                out[r, :n[r], h] = w @ vals
    return out


def _exact_verify(case, s):
    """Row by row: accept a child with probability min(1, p / q), else take max(p - q, 0), normalised, for p."""
    parents, tokens, n, u = s["parent"].tolist(), s["tokens"].tolist(), s["n"].tolist(), s["u"].double().tolist()
    paths, lengths, sampled = [], [], []
    for r in range(case["rows"]):
        if n[r] == 0:
            paths.append([-1] * case["nodes"])
            lengths.append(0)
            sampled.append(-1)
            continue
        path, node = [0], 0
        while True:
            p = s["target"][r, node].double().cpu().numpy()
            norm, moved = 1.0, False
            for c in range(node + 1, n[r]):
                if parents[r][c] != node:
                    continue
                t = tokens[r][c]
                if s["draft"] is None:
                    q = np.zeros_like(p)
                    q[t] = 1.0
                else:
                    q = s["draft"][r, node].double().cpu().numpy()
                if u[r][c] * q[t] < p[t] / norm:
                    path.append(c)
                    node, moved = c, True
                    break
                rest = np.maximum(p / norm - q, 0.0) if s["draft"] is not None else np.where(q > 0, 0.0, p / norm)
                if rest.sum() > 0:
                    p, norm = rest, rest.sum()
            if not moved:
                break
        below = np.cumsum(p)
        paths.append(path + [-1] * (case["nodes"] - len(path)))
        lengths.append(len(path))
        sampled.append(int(np.argmax(below > u[r][0] * below[-1])))
    return {"path": _i32(paths), "length": _i32(lengths), "token": _i32(sampled)}
