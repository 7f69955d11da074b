"""The barriers between one row tile's softmax and its products in the prompt attention, head size 128, as a model: every
order in which the products end and their arrivals come in.  Products end in the order of their issue; an arrival comes some
time after all products before it have ended, and no order holds between two arrivals.  A wait names the parity of a phase,
as an mbarrier's does."""
import itertools

import pytest


def programs(tiles, every_tile):
    """Softmax and products of segments of `tiles` token tiles.  every_tile: an arrival for the output after each tile's
    product, behind the next scores' own; otherwise one a segment.  "read" names the product that has to be done."""
    softmax, products = [], []
    scores = [(s, k) for s, n in enumerate(tiles) for k in range(n)]
    place = {x: i for i, x in enumerate(scores)}
    issued = 0
    done_at = {}  # (segment, tile): products issued up to its P V
    products += [("issue",), ("commit", "scores", 1)]
    issued = 1
    for (s, k) in scores:
        products.append(("wait", "weights", place[s, k] & 1))
        products.append(("issue",))
        issued += 1
        done_at[s, k] = issued
        last = k + 1 == tiles[s]
        if last:
            products.append(("commit", "output", issued))
        if place[s, k] + 1 < len(scores):
            products.append(("issue",))
            issued += 1
            products.append(("commit", "scores", issued))
        if every_tile and not last:
            products.append(("commit", "output", issued))
    def output(s):
        return [("wait", "output", (place[s, tiles[s] - 1] if every_tile else s) & 1), ("read", done_at[s, tiles[s] - 1])]

    for s, k in scores:
        softmax.append(("wait", "scores", place[s, k] & 1))
        if k:
            softmax.append(("read", done_at[s, k - 1]))  # the output may have to be rescaled
        elif s:
            softmax += output(s - 1)  # a segment's output is read when the next one's first weights are made
        softmax.append(("arrive", "weights"))
    softmax += output(len(tiles) - 1)
    return softmax, products


def fault(tiles, every_tile):
    """A state in which a read comes too early or nobody can go on, or None."""
    softmax, products = programs(tiles, every_tile)
    names = ["scores", "weights", "output"]
    start = (0, 0, 0, 0, (), (0, 0, 0))  # softmax, products, products issued and ended, arrivals on their way, phases
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        a, b, issued, ended, coming, done = state
        moved = []

        def arrive(name):
            return tuple(d + (n == name) for n, d in zip(names, done))

        if ended < issued:
            moved.append((a, b, issued, ended + 1, coming, done))
        for i, (name, needs) in enumerate(coming):
            if ended >= needs:
                moved.append((a, b, issued, ended, coming[:i] + coming[i + 1:], arrive(name)))
        for who, (at, prog) in enumerate(((a, softmax), (b, products))):
            if at == len(prog):
                continue
            op = prog[at]
            na, nb = (a + 1, b) if who == 0 else (a, b + 1)
            if op[0] == "wait":
                if done[names.index(op[1])] & 1 != op[2]:  # the current phase is not the awaited one
                    moved.append((na, nb, issued, ended, coming, done))
            elif op[0] == "arrive":
                moved.append((na, nb, issued, ended, coming, arrive(op[1])))
            elif op[0] == "issue":
                moved.append((na, nb, issued + 1, ended, coming, done))
            elif op[0] == "commit":
                moved.append((na, nb, issued, ended, tuple(sorted(coming + (op[1:],))), done))
            else:
                if ended < op[1]:
                    return state
                moved.append((na, nb, issued, ended, coming, done))
        if not moved and (a < len(softmax) or b < len(products)):
            return state
        for x in moved:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


@pytest.mark.parametrize("segments", [1, 2, 3])
def test_no_read_comes_too_early(segments):
    for tiles in itertools.product((1, 2, 3, 4), repeat=segments):
        assert fault(tiles, False) is None, tiles


def test_the_model_sees_a_phase_taken_for_the_next():
    """With an arrival for every tile, of which the softmax awaits a segment's last only, the parity may pass early."""
    assert fault((2,), True) is not None
    assert fault((3, 2), True) is not None
    assert fault((1, 1), True) is None  # nothing is left out
