"""Cases of the paged-cache operators: rotary positions, the append of a step's or a chunk's keys and values to a
cache in pages (rotated and, where the pages hold 8 bits, scaled on the way), and attention of one new token a
sequence over such a cache.

A serving loop runs, per layer, `paged_append` on the projections of the tokens it has, then `paged_decode` for the
sequences that generate.  `rope` is the rotation by itself, before `prompt` for instance, and with `inverse` its
backward pass.  A cache is a pool of pages, [pages, page, hkv, d] for keys and for values, and a table
[rows, most] with the page of each stretch of `page` positions of a sequence; `pos` is the position of the last
key, -1 for a sequence without any.

`run` computes each operator in its plain form, or with `own` set makes the package's calls.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one chat stream with a short history: a latency-bound call of every layer
        dict(name="decode_one_short", op="decode", rows=1, hq=16, hkv=8, d=256, page=16, win=0, lo=700, hi=700,
             bits=16, heads_first=False),
        # one stream with a long document behind it: the key axis is split over the card
        dict(name="decode_one_long", op="decode", rows=1, hq=32, hkv=4, d=128, page=64, win=0, lo=131071, hi=131071,
             bits=16, heads_first=False),
        # a serving batch with histories of every length, small pages
        dict(name="decode_batch", op="decode", rows=64, hq=32, hkv=8, d=128, page=16, win=0, lo=100, hi=16000,
             bits=16, heads_first=False),
        # a sliding layer: pages before the window have been given back
        dict(name="decode_window", op="decode", rows=48, hq=32, hkv=16, d=256, page=32, win=1024, lo=200, hi=60000,
             bits=16, heads_first=True),
        # a batch over 8-bit pages, groups of eight heads
        dict(name="decode_batch_8bit", op="decode", rows=64, hq=32, hkv=4, d=128, page=64, win=0, lo=500, hi=30000,
             bits=8, heads_first=False),
        # odd: seven sequences, one of them empty, groups of twelve heads, 8-bit pages of heads by tokens
        dict(name="decode_ragged_8bit", op="decode", rows=7, hq=24, hkv=2, d=256, page=128, win=0, lo=-1, hi=40001,
             bits=8, heads_first=True),
        # the step before decode_one_short
        dict(name="append_one", op="append", rows=1, hq=16, hkv=8, d=256, page=16, lo=701, hi=701, chunk=1,
             bits=16, rot=256, layout="half", heads_first=False),
        # a step of a batch into 8-bit pages, half of each head rotated in interleaved pairs
        dict(name="append_batch_8bit", op="append", rows=64, hq=32, hkv=8, d=128, page=16, lo=30, hi=9000, chunk=1,
             bits=8, rot=64, layout="interleaved", heads_first=False),
        # the chunks of five prompts together
        dict(name="append_chunk", op="append", rows=5, hq=32, hkv=8, d=128, page=64, lo=0, hi=20000, chunk=1637,
             bits=16, rot=128, layout="half", heads_first=False),
        # the rotation of one step's heads
        dict(name="rope_step", op="rope", n=64, heads=48, d=128, rot=128, layout="half", inverse=False, far=130000),
        # a long chunk, queries and keys of the interleaved projection rows
        dict(name="rope_chunk", op="rope", n=8192, heads=40, d=128, rot=128, layout="half", inverse=False, far=1000000),
        # the backward pass, a quarter of each head, odd length
        dict(name="rope_backward", op="rope", n=5003, heads=24, d=256, rot=64, layout="interleaved", inverse=True,
             far=32000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "append", "rope"])
    d = rng.choice([128, 256])
    if op == "rope":
        n, heads = _log(rng, 1, 12000), rng.randint(1, 64)
        while n * heads * d > 8192 * 40 * 128:
            n = n // 2
        return dict(op="rope", n=n, heads=heads, d=d, rot=16 * rng.randint(1, d // 16),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5, far=_log(rng, 100, 10 ** 9))
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    if hkv * group > 64:
        group = 2
    page, bits, heads_first = 2 ** rng.randint(4, 8), rng.choice([16, 16, 8]), rng.random() < 0.4
    rows = _log(rng, 1, 96)
    if op == "append":
        chunk = rng.choice([1, 1, _log(rng, 2, 2000)])
        while rows > 1 and rows * chunk * (hkv * group + 2 * hkv) * d > 5 * 1637 * 48 * 128:
            rows = max(1, rows // 2)
        while chunk > 1 and rows * chunk * (hkv * group + 2 * hkv) * d > 5 * 1637 * 48 * 128:
            chunk = chunk // 2
        lo = rng.randint(0, 300)
        return dict(op="append", rows=rows, hq=hkv * group, hkv=hkv, d=d, page=page, lo=lo,
                    hi=lo + _log(rng, 1, 20000), chunk=chunk, bits=bits, rot=rng.choice([0, d, d, d // 2, d // 4, 48]),
                    layout=rng.choice(["half", "interleaved"]), heads_first=heads_first)
    win = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    hi = _log(rng, 1, 131072)
    lo = rng.choice([-1, hi // 4, hi // 2, hi])
    span = min(win, hi + 1) if win else hi + 1
    while rows > 1 and (rows * span * hkv * d * bits // 4 > 2.1e9 or 4 * rows * span * hkv * group * d > 1.6e10):
        rows = max(1, rows // 2)
    return dict(op="decode", rows=rows, hq=hkv * group, hkv=hkv, d=d, page=page, win=win, lo=lo, hi=hi, bits=bits,
                heads_first=heads_first)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, rows):
    """`rows` whole numbers from lo to hi, evenly apart."""
    return [lo + (hi - lo) * i // max(1, rows - 1) for i in range(rows)] if rows > 1 else [hi]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(shape, gen, rms=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, rms, generator=gen)


def _pages(count, case, gen, rms):
    """A pool of pages, stored token by token or head by head, and the scale of each head's values."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    shape = (count, hkv, page, d) if case["heads_first"] else (count, page, hkv, d)
    pool, scale = _normal(shape, gen, rms if case["bits"] == 16 else 448 / 5.0), None
    if case["bits"] == 8:       # values up to five deviations fill the type's range
        scale = rms * 5.0 / 448 * torch.linspace(0.9, 1.1, hkv, device="cuda")
        pool = pool.clamp_(-448, 448).to(torch.float8_e4m3fn)
    return (pool.transpose(1, 2) if case["heads_first"] else pool), scale


def _table(lasts, firsts, page, r):
    """The page of each stretch of each sequence: a shuffled pool, -1 where a sequence has no key or none any more."""
    most = max(1, max(last // page + 1 for last in lasts))
    live = [(i, j) for i, (a, b) in enumerate(zip(firsts, lasts)) for j in range(a // page, b // page + 1)]
    ids = list(range(len(live) + 3))
    r.shuffle(ids)
    table = [[-1] * most for _ in lasts]
    for (i, j), page_id in zip(live, ids):
        table[i][j] = page_id
    return table, len(ids)


def prepare(case, seed):
    r = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed * 1013 + 29)
    s = dict(case)
    d = case["d"]
    if case["op"] == "rope":
        n, heads = case["n"], case["heads"]
        s["x"] = _normal((n, heads, d), gen)
        start = r.randint(0, case["far"])
        s["pos"] = _i32(list(range(start, start + n)))
        s["inv_freq"] = _frequencies(case["rot"])
        s["out"] = torch.empty_like(s["x"])
        return s
    rows, hq, hkv, page = case["rows"], case["hq"], case["hkv"], case["page"]
    last = _spread(case["lo"], case["hi"], rows)
    r.shuffle(last)
    if case["op"] == "append":
        ends = [p + case["chunk"] - 1 for p in last]
        table, count = _table(ends, last, page, r)
        s["pos"] = _i32([p + i for p in last for i in range(case["chunk"])])
        s["row"] = None if case["chunk"] == 1 else _i32([i for i in range(rows) for _ in range(case["chunk"])])
        n = rows * case["chunk"]
        s["src"] = _normal((n, (hq + 2 * hkv) * d), gen)
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
        s["inv_freq"] = _frequencies(case["rot"]) if case["rot"] else None
    else:
        table, count = _table(last, [max(0, p - case["win"] + 1) if case["win"] else 0 for p in last], page, r)
        s["pos"], s["last"] = _i32(last), last
        s["q"] = _normal((rows, hq, d), gen)
        s["scale"] = 1.0 if d == 256 else 1.0 / math.sqrt(d)
    rms = 0.1 if d == 256 else 1.0
    s["k_pages"], s["k_scale"] = _pages(count, case, gen, rms)
    s["v_pages"], s["v_scale"] = _pages(count, case, gen, 1.0)
    s["table"] = _i32(table)
    if case["op"] == "decode":       # a peaked key a sequence and head: one along a query, at a score of about 10
        row = [i for i, p in enumerate(last) if p >= 0]
        if row:
            at = [r.randint(max(0, last[i] - case["win"] + 1) if case["win"] else 0, last[i]) for i in row]
            ids = [table[i][p // page] for i, p in zip(row, at)]
            rise = (0.04 if d == 256 else 0.9) * s["q"][row][:, ::hq // hkv].float()
            if case["bits"] == 8:
                rise = (rise / s["k_scale"][:, None]).clamp(-448, 448)
            s["k_pages"][torch.tensor(ids, device="cuda"), torch.tensor([p % page for p in at], device="cuda")] = \
                rise.to(s["k_pages"].dtype)
    return s


def _frequencies(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if s["op"] == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    if s["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_decode(s) if own else _plain_decode(s)


def _own_rope(s):
    import sliding_window_gqa_gb300 as wa
    return wa.rope(s["x"], s["pos"], s["inv_freq"], layout=s["layout"], inverse=s["inverse"], out=s["out"])


def _own_append(s):
    import sliding_window_gqa_gb300 as wa
    wa.paged_append(s["src"], s["pos"], s["q_out"], s["k_pages"], s["v_pages"], s["table"], row=s["row"],
                    inv_freq=s["inv_freq"], layout=s["layout"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _own_decode(s):
    import sliding_window_gqa_gb300 as wa
    return wa.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["pos"], win=s["win"], scale=s["scale"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"])


def _turned(x, pos, inv_freq, layout, inverse=False):
    """x [n, heads, d] in 32 bits with its first 2 len(inv_freq) dims rotated; angles in 64."""
    if inv_freq is None:
        return x.float()
    angle = pos.double()[:, None] * inv_freq.double()
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sn = -sn
    R = 2 * inv_freq.numel()
    y = x.float()
    if layout == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        return torch.cat([a * c - b * sn, b * c + a * sn, y[..., R:]], -1)
    a, b = y[..., 0:R:2], y[..., 1:R:2]
    return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), y[..., R:]], -1)


def _plain_rope(s):
    return _turned(s["x"], s["pos"], s["inv_freq"], s["layout"], s["inverse"]).to(torch.bfloat16)


def _plain_append(s):
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    x = s["src"].view(-1, hq + 2 * hkv, d)
    qk = _turned(x[:, :hq + hkv], s["pos"], s["inv_freq"], s["layout"])
    s["q_out"].copy_(qk[:, :hq])
    pos = s["pos"].long()
    row = torch.arange(pos.numel(), device=pos.device) if s["row"] is None else s["row"].long()
    at = s["table"][row, pos // page].long(), pos % page
    for new, pages, scale in ((qk[:, hq:], s["k_pages"], s["k_scale"]), (x[:, hq + hkv:].float(), s["v_pages"], s["v_scale"])):
        if scale is not None:
            new = (new / scale[:, None]).clamp(-448, 448)
        pages[at] = new.to(pages.dtype)
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _plain_decode(s):
    """Sequence by sequence: the visible pages in 32 bits, and the softmax over their keys."""
    hq, hkv, d, page, win = s["hq"], s["hkv"], s["d"], s["page"], s["win"]
    out = torch.zeros_like(s["q"])
    for i, last in enumerate(s["last"]):
        if last < 0:
            continue
        first = max(0, last - win + 1) if win else 0
        ids = s["table"][i, first // page:last // page + 1].long()
        skip = first - first // page * page
        k, v = (pages[ids].float().flatten(0, 1)[skip:skip + last - first + 1] for pages in (s["k_pages"], s["v_pages"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
        w = torch.matmul(s["q"][i].float().view(hkv, hq // hkv, d), k.permute(1, 2, 0)) * s["scale"]
        w = (w - w.amax(-1, keepdim=True)).exp()
        o = torch.matmul(w, v.transpose(0, 1)) / w.sum(-1, keepdim=True)
        out[i] = o.view(hq, d).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    d = case["d"]
    if case["op"] == "rope":
        return {"bytes": 4 * case["n"] * case["heads"] * d, "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    hq, hkv, size = case["hq"], case["hkv"], case["bits"] // 8
    if case["op"] == "append":
        n = case["rows"] * case["chunk"]
        return {"bytes": n * d * (2 * (2 * hq + 2 * hkv) + 2 * hkv * size), "flops": 3 * n * (hq + hkv) * case["rot"]}
    last = _spread(case["lo"], case["hi"], case["rows"])
    keys = sum(min(p + 1, case["win"]) if case["win"] else p + 1 for p in last)
    return {"bytes": 2 * keys * hkv * d * size + 4 * case["rows"] * hq * d, "flops": 4 * keys * hq * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rotate64(s["x"], s["pos"], s["inv_freq"], case["layout"], -1.0 if case["inverse"] else 1.0)
    if case["op"] == "append":
        return _append64(case, s)
    return _decode64(case, s)


def _rotate64(x, pos, inv_freq, layout, sign=1.0):
    """Each pair as a complex number times e^(i pos w)."""
    y = x.double().clone()
    w = inv_freq.double()
    pairs = w.numel()
    by = torch.polar(torch.ones_like(pos, dtype=torch.float64)[:, None].expand(-1, pairs),
                     sign * torch.outer(pos.double(), w))[:, None, :]
    one, two = (slice(0, pairs), slice(pairs, 2 * pairs)) if layout == "half" else (slice(0, 2 * pairs, 2),
                                                                                   slice(1, 2 * pairs, 2))
    z = torch.complex(y[..., one], y[..., two]) * by
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _append64(case, s):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    heads = s["src"].double().view(-1, hq + 2 * hkv, d)
    q, k, v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
    if case["rot"]:
        q, k = (_rotate64(x, s["pos"], s["inv_freq"], case["layout"]) for x in (q, k))
    result = {"q": q}
    where = s["pos"].long()
    seq = where.new_tensor(range(case["rows"])).repeat_interleave(case["chunk"])
    slot = s["table"].long()[seq, torch.div(where, page, rounding_mode="floor")] * page + where % page
    for name, new, scale in (("k", k, s["k_scale"]), ("v", v, s["v_scale"])):
        pool = s[name + "_pages"].double().reshape(-1, hkv, d).clone()
        if scale is not None:
            new = torch.clip(new / scale.double()[None, :, None], -448.0, 448.0)
        pool.index_copy_(0, slot, new)
        result[name] = pool.view(-1, page, hkv, d)
    return result


def _decode64(case, s):
    """Head by head over the positions that are seen, each looked up by its page."""
    hq, hkv, d, page, win = case["hq"], case["hkv"], case["d"], case["page"], case["win"]
    out = torch.zeros((case["rows"], hq, d), dtype=torch.float64, device="cuda")
    for i, p in enumerate(s["pos"].tolist()):
        at = torch.arange(max(0, p - win + 1) if win else 0, p + 1, device="cuda")
        if not at.numel():
            continue
        where = s["table"][i].long()[at // page], at % page
        for g in range(hkv):
            k, v = s["k_pages"][:, :, g][where].double(), s["v_pages"][:, :, g][where].double()
            if case["bits"] == 8:
                k, v = k * s["k_scale"][g].double(), v * s["v_scale"][g].double()
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                weight = torch.softmax(k @ s["q"][i, h].double() * (1.0 if d == 256 else 1.0 / math.sqrt(d)), 0)
                out[i, h] = weight @ v
    return out
