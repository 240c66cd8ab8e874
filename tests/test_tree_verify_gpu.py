"""Verification of drafted tokens on the GPU against the float64 definition: every whole number equal.

The kernel's sums carry about 46 bits and the definition's 53, so they could part only where a random number lies
within about 2^-40 of a border, which the cases' 2^-24-spaced numbers do by chance in fewer than one run in a
thousand million; borders that are hit exactly (sums of few powers of two) are exact in both.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import wa_synth
from _util import ensure_built
from oracle import tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def make(rows, nodes, vocab, seed, kind="random", draft=True, noise=1.0, peak=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((rows, nodes, vocab), generator=gen, device="cuda") * peak
    target = torch.softmax(logits, -1)
    q = torch.softmax(logits + noise * torch.randn((rows, nodes, vocab), generator=gen, device="cuda"), -1)
    parent = torch.tensor([wa_synth.draft_tree(kind, nodes, seed + r) for r in range(rows)], dtype=torch.int32,
                          device="cuda")
    at = parent.long().clamp_min(0)
    row = torch.arange(rows, device="cuda")[:, None]
    tokens = torch.multinomial(q[row, at].view(-1, vocab), 1, generator=gen).view(rows, nodes).int()
    u = torch.rand((rows, nodes), generator=gen, device="cuda")
    return dict(target=target, draft=q if draft else None, parent=parent, tokens=tokens, u=u)


def both(wa, c, n=None, **kw):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    nt = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    path, length, token = wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"], n=nt, ws=ws,
                                         **kw)
    d = None if c["draft"] is None else c["draft"].cpu().numpy()
    want = tree.verify(c["target"].cpu().numpy(), d, c["parent"].tolist(), c["tokens"].tolist(), c["u"].cpu().numpy(), n)
    assert (path.tolist(), length.tolist(), token.tolist()) == want
    return wa.status(ws), want


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "points"])
@pytest.mark.parametrize("rows,nodes,vocab,kind", [
    (1, 1, 1, "chain"), (2, 2, 2, "chain"), (3, 9, 31, "random"), (5, 13, 1000, "bushy"), (2, 8, 32768, "chain"),
    (17, 26, 1025, "bushy"), (1, 128, 511, "random"), (4, 33, 10007, "random"), (3, 6, 100003, "random"),
    (2, 5, 262144, "bushy"), (40, 4, 4099, "chain"),
])
def test_equal_to_the_definition(wa, rows, nodes, vocab, kind, draft):
    for noise in (0.3, 2.0):
        st, want = both(wa, make(rows, nodes, vocab, seed=nodes + vocab, kind=kind, draft=draft, noise=noise))
        assert st == 0


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "points"])
def test_rejections_all_the_way(wa, draft):
    """Drafts that the target holds to be unlikely: every child is dropped, several rounds at one node."""
    c = make(6, 12, 5000, seed=3, kind="flat", draft=draft, noise=4.0)
    c["parent"][:, 1:] = 0
    c["u"][:, 1:] = 1.0 - 2.0 ** -24
    st, (path, length, token) = both(wa, c)
    assert st == 0 and min(length) == 1


def test_few_tokens_with_weight(wa):
    """Distributions on a handful of tokens; the draft's on the same and on others; p = q."""
    rows, nodes, V = 8, 5, 3000
    c = make(rows, nodes, V, seed=7)
    keep = torch.zeros(V, device="cuda")
    keep[[0, 17, 1023, 1024, 2999]] = 1.0
    c["target"] = c["target"] * keep
    c["target"] /= c["target"].sum(-1, keepdim=True)
    both(wa, c)
    c["draft"] = c["target"].clone()
    both(wa, c)
    c["draft"] = c["draft"] * 0
    both(wa, c)


def test_borders_that_are_hit(wa):
    """Power-of-two weights and random numbers on their borders: strict comparisons, exact sums."""
    V = 8
    p = torch.tensor([0.25, 0, 0.25, 0.125, 0.125, 0, 0.25, 0], device="cuda")
    us = [0.0, 0.125, 0.25, 0.5, 0.625, 0.75, 1.0 - 2.0 ** -24, 1.0, float("nan"), -0.5]
    rows = len(us)
    c = dict(target=p.expand(rows, 1, V).contiguous(), draft=None,
             parent=torch.full((rows, 1), -1, dtype=torch.int32, device="cuda"),
             tokens=torch.zeros((rows, 1), dtype=torch.int32, device="cuda"),
             u=torch.tensor(us, device="cuda")[:, None].contiguous())
    _, (_, _, token) = both(wa, c)
    assert token == [0, 0, 2, 3, 4, 6, 6, 6, 6, 0]
    # a test of u q < p at equality drops the child, u = 0 keeps one with weight and drops one without
    q = torch.full((V,), 0.125, device="cuda")
    c = dict(target=p.expand(3, 2, V).contiguous(), draft=q.expand(3, 2, V).contiguous(),
             parent=torch.tensor([[-1, 0]] * 3, dtype=torch.int32, device="cuda"),
             tokens=torch.tensor([[0, 3], [0, 0], [0, 1]], dtype=torch.int32, device="cuda"),
             u=torch.tensor([[0.3, 1.0], [0.3, 0.0], [0.3, 0.0]], device="cuda"))
    _, (_, length, _) = both(wa, c)
    assert length == [1, 2, 1]


def test_values_that_are_no_probabilities(wa):
    c = make(4, 6, 700, seed=2)
    c["target"][0, :, 5] = float("nan")
    c["target"][1, :, ::2] = -0.25
    c["target"][2, :, 9] = float("inf")
    c["draft"][3, :, 4] = float("nan")
    c["draft"][3, :, 8] = 3.0
    st, _ = both(wa, c)
    assert st == 0
    c["target"][1] = float("nan")
    c["u"][1, 1:] = 0.5
    st, (_, length, token) = both(wa, c)
    assert st == wa.WA_STATUS_NO_MASS and length[1] == 1 and token[1] == -1


def test_ragged_rows_and_status(wa):
    c = make(6, 7, 600, seed=9, kind="bushy")
    st, (path, length, token) = both(wa, c, n=[0, 1, 2, 4, 6, 7])
    assert st == 0 and length[0] == 0 and token[0] == -1 and path[0] == [-1] * 7
    for n in ([8, 1, 2, 4, 6, 7], [-3, 1, 2, 4, 6, 7]):
        assert both(wa, c, n=n)[0] == wa.WA_STATUS_BAD_TREE
    c["tokens"][4, 1] = 600
    c["tokens"][5, 2] = -1
    assert both(wa, c)[0] == wa.WA_STATUS_BAD_TREE
    c = make(6, 7, 600, seed=9, kind="bushy")
    c["tokens"][:, 0] = -5                    # not read
    assert both(wa, c)[0] == 0
    c["parent"][2, 3] = 5
    assert both(wa, c)[0] == wa.WA_STATUS_BAD_TREE


@pytest.mark.parametrize("vocab", [1001, 4096])
def test_strides(wa, vocab):
    """Probabilities cut from wider rows (also off every 16-byte border), nodes before rows, outputs given."""
    c = make(5, 6, vocab, seed=5)
    wide = torch.full((5, 6, vocab + 9), float("nan"), device="cuda")
    t = wide[:, :, 3:vocab + 3]
    t.copy_(c["target"])
    swapped = torch.zeros((6, 5, vocab), device="cuda").transpose(0, 1)
    swapped.copy_(c["draft"])
    want = wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"])
    outs = [torch.full(s, 99, dtype=torch.int32, device="cuda") for s in ((5, 6), (5,), (5,))]
    got = wa.tree_verify(t, c["parent"], c["tokens"], c["u"], draft=swapped, path=outs[0], length=outs[1],
                         token=outs[2])
    for a, b, o in zip(got, want, outs):
        assert torch.equal(a, b) and a is o


def test_streams_and_graphs(wa):
    cs = [make(9, 8, 20011, seed=s) for s in (1, 2)]
    want = [wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"]) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"], stream=s)
               for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = cs[0]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    outs = dict(path=torch.zeros((9, 8), dtype=torch.int32, device="cuda"),
                length=torch.zeros(9, dtype=torch.int32, device="cuda"),
                token=torch.zeros(9, dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"], ws=ws, stream=streams[0], **outs)
    for _ in range(3):
        c["u"].copy_(torch.rand_like(c["u"]))
        g.replay()
        torch.cuda.synchronize()
        p = tree.verify(c["target"].cpu().numpy(), c["draft"].cpu().numpy(), c["parent"].tolist(),
                        c["tokens"].tolist(), c["u"].cpu().numpy())
        assert (outs["path"].tolist(), outs["length"].tolist(), outs["token"].tolist()) == p


def test_kept_tokens_are_distributed_as_the_target(wa):
    """40,000 rows that draft two children from q: the token that follows has the target's distribution.  A share's
    standard deviation is at most 0.0025; held to four of them."""
    rows, V = 40000, 12
    gen = torch.Generator(device="cuda").manual_seed(4)
    p, q = torch.softmax(torch.randn((2, V), generator=gen, device="cuda") * 1.5, -1)
    tokens = torch.multinomial(q.expand(rows, V), 3, replacement=True, generator=gen).int()
    u = torch.rand((rows, 3), generator=gen, device="cuda")
    parent = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda").repeat(rows, 1)
    path, length, token = wa.tree_verify(p.expand(rows, 3, V).contiguous(), parent, tokens, u,
                                         draft=q.expand(rows, 3, V).contiguous())
    kept = tokens.gather(1, path[:, 1:2].long().clamp_min(0))[:, 0]
    after = torch.where(length > 1, kept, token)
    share = torch.bincount(after, minlength=V).double() / rows
    assert (share - p.double()).abs().max() < 4 * np.sqrt(0.25 / rows)


def test_result_does_not_depend_on_the_rows_around_it(wa):
    """The same row alone, among 40, 80 and 400: clusters of 8, 4, 2 and 1 CTAs sum in one order."""
    c = make(8, 12, 30011, seed=21, kind="bushy", noise=1.5)
    for draft in (c["draft"], None):
        want = [t.tolist() for t in wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=draft)]
        for times in (5, 10, 50):
            rep = lambda t: t.repeat(times, *[1] * (t.dim() - 1))   # noqa: E731
            got = wa.tree_verify(rep(c["target"]), rep(c["parent"]), rep(c["tokens"]), rep(c["u"]),
                                 draft=None if draft is None else rep(draft))
            assert [t.tolist() for t in got] == [w * times for w in want]
        one = wa.tree_verify(*[c[x][3:4].contiguous() for x in ("target", "parent", "tokens", "u")],
                             draft=None if draft is None else draft[3:4].contiguous())
        assert [t.tolist() for t in one] == [w[3:4] for w in want]


def test_a_single_rows_status(wa):
    """One row clears the workspace's status itself: whatever a call before left, or fresh memory holds."""
    good = make(1, 6, 3001, seed=8)
    bad = dict(good, tokens=good["tokens"].clone(), target=torch.zeros_like(good["target"]))
    bad["tokens"][0, 3] = -5
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    for c, want in ((good, 0), (bad, wa.WA_STATUS_BAD_TREE | wa.WA_STATUS_NO_MASS), (good, 0)):
        path, length, token = wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"], ws=ws)
        assert wa.status(ws) == want
        ref = tree.verify(c["target"].cpu().numpy(), c["draft"].cpu().numpy(), c["parent"].tolist(), c["tokens"].tolist(),
                          c["u"].cpu().numpy())
        assert (path.tolist(), length.tolist(), token.tolist()) == ref


def near(rows, V, k, seed, device="cuda"):
    """A target and a draft within 1e-8 to 1e-5 of it (relative to each token's own probability), and k siblings below
    node 0 that hold tokens of which the draft has more: all are dropped, and what is left of the target is small."""
    gen = torch.Generator().manual_seed(seed)
    p = torch.softmax(2.0 * torch.randn((rows, V), generator=gen, dtype=torch.float64), -1).float()
    size = 10.0 ** (-8.0 + 3.0 * torch.rand((rows, 1), generator=gen, dtype=torch.float64))
    q = (p.double() * (1.0 + size * torch.randn((rows, V), generator=gen, dtype=torch.float64))).float()
    over = (q > p).double() + 1e-30
    tokens = torch.cat([torch.zeros((rows, 1), dtype=torch.int64), torch.multinomial(over, k, True, generator=gen)], 1)
    u = torch.full((rows, k + 1), 1.0 - 2.0 ** -24)
    u[:, 0] = torch.rand(rows, generator=gen)
    parent = torch.zeros((rows, k + 1), dtype=torch.int32)
    parent[:, 0] = -1
    c = dict(target=p[:, None].expand(rows, k + 1, V), draft=q[:, None].expand(rows, k + 1, V), parent=parent,
             tokens=tokens.int(), u=u)
    return {n: t.contiguous().to(device) for n, t in c.items()}


def dropped(c, tol):
    """The definition in float64 for rows of near(): what is left of the target once every child is dropped, and the
    rows of which it is sure, if weights, sums and S q may be off by tol, that all of them are."""
    p, q = c["target"][:, 0].double(), c["draft"][:, 0].double()
    rows, k = p.shape[0], c["u"].shape[1] - 1
    row = torch.arange(rows, device=p.device)
    w, S = p, torch.zeros(rows, 1, dtype=torch.float64, device=p.device)
    s = torch.ones_like(S)
    sure = torch.ones(rows, dtype=torch.bool, device=p.device)
    for i in range(1, k + 1):
        x = c["tokens"][:, i].long()
        test = c["u"][:, i].double() * q[row, x] * s[:, 0] - w[row, x]
        sure &= (test > tol) | ((test >= 0) & ((p - S * q)[row, x] < -tol * p[row, x]))
        left = (p - (S + s) * q).clamp_min(0)
        mass = left.sum(1, keepdim=True)
        near_0 = ((p - (S + s) * q).abs() <= tol * p).any(1) & (S + s != 1)[:, 0]
        sure &= (mass[:, 0] > tol) | ((mass[:, 0] == 0) & ~near_0)
        on = mass > 0
        w, S, s = torch.where(on, left, w), torch.where(on, S + s, S), torch.where(on, mass, s)
    return w, sure


@pytest.mark.parametrize("V,k,rows", [(5, 2, 3000), (5, 5, 3000), (31, 3, 3000), (130, 2, 2000), (1003, 4, 1500),
                                      (20011, 3, 150)])
def test_little_is_left_of_the_target(wa, V, k, rows):
    """Draft probabilities next to the target's: the residual that the last token is drawn from is 1e-8 to 1e-5.

    A weight W(x) = p(x) - S q(x) of the kernel is off by at most 2^-45 p(x) (its low part, at most 2^-23 p(x), takes six
    fp32 roundings) and by q(x) times S's error, 2^-47 a drop (S's low part the same way); the sums of what is left add
    2^-38 of sums below 2^-16 at most.  Running sums are off by less than 2^-45 + k 2^-47 + 2^-54 < 2^-43, the random
    number's place the same, so the kernel's token is one whose stretch of the definition's running sum comes within
    2^-41 of the place, and has weight there."""
    tol = 2.0 ** -41
    c = near(rows, V, k, seed=V + k)
    path, length, token = wa.tree_verify(c["target"], c["parent"], c["tokens"], c["u"], draft=c["draft"])
    w, sure = dropped(c, tol)
    assert sure.double().mean() > 0.5
    assert (length[sure] == 1).all()
    run = w.cumsum(1)
    place = c["u"][:, :1].double() * run[:, -1:]
    assert (token[sure] >= 0).all()
    at = token.long().clamp_min(0)[:, None]
    end, own = run.gather(1, at), w.gather(1, at)
    good = ((end - own <= place + tol) & (end > place - tol) & (own > 0))[:, 0]
    assert good[sure].all(), f"{(~good[sure]).sum().item()} of {sure.sum().item()}"


def cluster(rows, sms):
    """CTAs a row: the most of 8, 4, 2, 1 with which the rows have at most 4 CTAs an SM."""
    return next(cl for cl in (8, 4, 2, 1) if cl == 1 or 4 * sms // rows >= cl)


def test_every_cluster_size(wa):
    """The same eight rows among as many as bring clusters of 8, 4, 2 and 1 CTAs, on both sides of each border."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = make(8, 10, 4099, seed=23, kind="bushy", noise=1.5)
    seen = set()
    for draft in (True, False):
        _, want = both(wa, c if draft else dict(c, draft=None))
        for rows in (sms // 2, sms // 2 + 1, sms, sms + 1, 2 * sms - 3, 2 * sms, 2 * sms + 1, 4 * sms):
            seen.add(cluster(rows, sms))
            at = torch.arange(rows, device="cuda") % 8
            got = wa.tree_verify(*[c[x][at] for x in ("target", "parent", "tokens", "u")],
                                 draft=c["draft"][at] if draft else None)
            for g, w in zip(got, want):
                assert g.tolist() == [w[i] for i in at.tolist()], rows
    assert seen == {8, 4, 2, 1}


def test_vocabularies_past_32_bits_are_refused(wa):
    """Not taken modulo 2^32.  (17 GB that nothing reads.)"""
    target = torch.empty((1, 1, 2 ** 32 + 8), device="cuda")
    one = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        wa.tree_verify(target, one, one, one.float())
    with pytest.raises(wa.WAError):
        wa.tree_verify(target[:, :, :2 ** 24 + 1].contiguous(), one, one, one.float())
