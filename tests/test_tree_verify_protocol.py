"""How the CTAs of a verification's cluster leave, as a model on the CPU: every order of events, waits that run out included.

The CTAs of a row make the same passes.  In each a CTA stores its sums to every CTA of the cluster (a store arrives some
time later, counted on the receiver's barrier), then waits for all of them; a wait that runs out makes the CTA late, and
a late one sends nothing more.  A store must not arrive at a CTA that has left.  A store takes far less time than a wait's
limit: a CTA's wait runs out only after its own stores of that pass have arrived, and a wait that began when every CTA had
stopped sending only after all have.  Another CTA's store may be under way when a wait runs out.
"""
from __future__ import annotations

import pytest

SEND, WAIT, MEET, LEAVE, GONE = range(5)


def lost_stores(ctas: int, passes: int, meet: bool) -> int:
    """States in which a store finds its CTA gone.  meet: as the kernel does, a CTA that is through all passes announces it
    and leaves, and a late one stays until all have announced that they are through or late; else a late one goes on by
    itself.  Either way it then waits once more for the pass that it gave up on."""
    # a CTA: (what it does next, pass, late); a store under way: (from, to, pass); what has arrived: (to, pass) -> from
    start = (tuple((SEND, 0, False) for _ in range(ctas)), frozenset(), frozenset())
    todo, known, lost = [start], {start}, 0
    while todo:
        state, flying, landed = todo.pop()

        def step(i, new, flying=flying, landed=landed):
            nxt = (state[:i] + (new,) + state[i + 1:], flying, landed)
            if nxt not in known:
                known.add(nxt)
                todo.append(nxt)

        for m in flying:
            if state[m[1]][0] == GONE:
                lost += 1
            step(0, state[0], flying=flying - {m}, landed=landed | {m})
        for i, (do, k, late) in enumerate(state):
            through = all((j, i, k) in landed for j in range(ctas))
            if do == SEND:
                step(i, (WAIT, k, False), flying=flying | {(i, j, k) for j in range(ctas)})
            elif do == WAIT:
                if through:
                    step(i, (SEND, k + 1, False) if k + 1 < passes else (GONE, k, False))
                elif not any(m[0] == i for m in flying):
                    step(i, (MEET if meet else LEAVE, k, True))
            elif do == MEET:
                if all(s[0] in (MEET, LEAVE, GONE) for s in state):
                    step(i, (LEAVE, k, late))
            elif do == LEAVE and (through or not meet or not flying):
                step(i, (GONE, k, late))
    return lost


@pytest.mark.parametrize("ctas,passes", [(2, 1), (2, 2), (2, 3), (3, 1), (3, 2)])
def test_no_store_finds_its_cta_gone(ctas, passes):
    assert lost_stores(ctas, passes, meet=True) == 0


def test_leaving_one_by_one_would_lose_stores():
    assert lost_stores(2, 2, meet=False) > 0
