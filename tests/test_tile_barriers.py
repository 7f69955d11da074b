"""The barriers between the softmax and the two product warps of the tile attention kernel, as a model: every interleaving
of the three ends.  A wait names the parity of a phase, as an mbarrier's does, so whoever falls two phases behind takes
the wrong phase for the awaited one."""
import itertools

import pytest


def programs(tiles, per_group):
    """The roles' arrivals and waits for segments of `tiles` token tiles; tile k belongs to group k % 2.  per_group: a product
    warp waits for the queries of its group's segments; otherwise for those of every segment, on one barrier."""
    starts = [0, *itertools.accumulate(tiles)]
    softmax, products = [], [[], []]
    phase = [0, 0]
    for s, n in enumerate(tiles):
        own = [[k for k in range(starts[s], starts[s] + n) if k % 2 == g] for g in (0, 1)]
        softmax += [("arrive", ("queries", g)) for g in (0, 1) if own[g]] if per_group else [("arrive", ("queries", 0))]
        for k in range(starts[s], starts[s] + n):
            softmax += [("wait", ("scores", k % 2), k // 2 & 1), ("arrive", ("weights", k % 2))]
        softmax += [("wait", ("output", g), own[g][-1] // 2 & 1) for g in (0, 1) if own[g]]
        for g in (0, 1):
            if not per_group:
                products[g].append(("wait", ("queries", 0), s & 1))
            elif own[g]:
                products[g].append(("wait", ("queries", g), phase[g]))
                phase[g] ^= 1
            for k in own[g]:
                products[g] += [("arrive", ("scores", g)), ("wait", ("weights", g), k // 2 & 1), ("arrive", ("output", g))]
    return [softmax, *products]


def stuck(progs):
    """A state that no role can leave although one has not ended, or None."""
    barriers = sorted({op[1] for p in progs for op in p})
    start = ((0,) * len(progs), (0,) * len(barriers))
    seen, todo = {start}, [start]
    while todo:
        at, done = todo.pop()
        moved = False
        for i, p in enumerate(progs):
            if at[i] == len(p):
                continue
            kind, name, *parity = p[at[i]]
            j = barriers.index(name)
            if kind == "wait" and done[j] & 1 == parity[0]:  # the current phase has the awaited one's parity: not complete
                continue
            moved = True
            state = (at[:i] + (at[i] + 1,) + at[i + 1:], done[:j] + (done[j] + (kind == "arrive"),) + done[j + 1:])
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(a < len(p) for a, p in zip(at, progs)):
            return at
    return None


@pytest.mark.parametrize("segments", [1, 2, 3, 4, 5])
def test_no_interleaving_is_stuck(segments):
    for tiles in itertools.product((1, 2, 3), repeat=segments):
        assert stuck(programs(tiles, True)) is None, tiles


def test_the_model_sees_a_warp_that_falls_behind():
    """Waiting for the queries of every segment leaves a warp behind that has no tile in some of them."""
    assert stuck(programs((1, 1, 1, 1, 1), False)) is not None
    assert stuck(programs((2, 2, 2), False)) is None
