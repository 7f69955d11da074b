"""The offsets of the prompt attention's weights in 32-bit arithmetic, restated on the CPU: a row's scores come in tiles of 128,
weights are powers of two under an offset near the largest score so far, and fp16 has to hold them (for bf16 their sums have
to stay below 1).  The restatement follows csrc/prompt.cuh's arithmetic step by step, with an offset of one number as well,
for what that cannot do."""
import math

import numpy as np
import pytest

F = np.float32
TYPES = {"f16": (F(8), F(60000)), "bf16": (F(-25), F(60000 / 2 ** 33))}  # the largest weight's exponent, a tile's most
FAR, TILE = F(2 ** 20), 128
NINF = F(-math.inf)


def fma(a, b, c):
    """One rounding: a product of two 32-bit numbers is exact in 64 bits."""
    with np.errstate(invalid="ignore", over="ignore"):
        return (np.asarray(a, np.float64) * np.float64(b) + np.float64(c)).astype(F)


def ex2(x):
    """The device's exponential: numbers below 2^-126 become 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.exp2(np.asarray(x, np.float64)).astype(F)
    return np.where(y < F(2.0 ** -126), F(0), y)


def row(scores, scale, kind, two=True):
    """(weights, sum, offset as (number, rest), most passes over a tile), or None if a tile's passes do not end."""
    UP, MOST = TYPES[kind]
    f = F(scale * 1.4426950408889634)
    size, over = F(abs(f)), F(1) / f
    m, lo, total, weights, most, hard, less = NINF, F(0), F(0), np.zeros(0, F), 0, False, F(0)
    with np.errstate(invalid="ignore", over="ignore"):
        for at in range(0, len(scores), TILE):
            s, limit, passes = scores[at:at + TILE], MOST, 0
            top = (s if f >= 0 else -s).max()
            if m == NINF or hard:
                first = F(top * size - UP) if m == NINF else m
                if two and abs(first) > FAR / F(2) and first != NINF:
                    limit = F(-1)
                else:
                    m, less = first, F(0) if first == NINF else first
            while True:
                passes += 1
                w = ex2(fma(s, f, -less))
                if not w.sum(dtype=F) > limit:
                    break
                if passes == 4:
                    return None
                nm, nl, a = F(top * size), F(0), F(1)
                if two and abs(nm) > FAR and nm != NINF:
                    nl = F(fma(top, size, -nm))
                    if abs(nl) < FAR / F(16):
                        nl = F(nl - UP)
                else:
                    nm = F(nm - UP)
                up = F(F(nm - m) + F(nl - lo))
                if nm > NINF and not up <= 0:
                    a, m, lo = ex2(-up), nm, nl
                total, weights = F(total * a), (weights * a).astype(F)
                hard, less = two and abs(m) > FAR, m
                if hard:  # the tile's exponents, over f, take its scores' place
                    s, less = ((fma(s, f, -m) - lo) * over).astype(F), F(0)
                if two:
                    limit = F(math.inf)
            most = max(most, passes)
            total, weights = F(total + w.sum(dtype=F)), np.concatenate([weights, w])
    return weights, total, (m, lo), most


def cases(size, seed):
    """Rows of scores near `size`, exact in 32 bits."""
    g = np.random.default_rng(seed)
    n = 400
    yield np.full(n, size * g.uniform(0.5, 1), F)                                    # all alike
    yield (size * g.uniform(0.5, 1, n)).astype(F)                                    # all different
    yield (size * (1 + g.integers(-4, 5, n) * 2.0 ** -23)).astype(F)                 # a few last places apart
    yield (-size * g.uniform(0.5, 1, n)).astype(F)
    yield (size * np.linspace(-1, 1, n)).astype(F)                                   # rising
    yield (size * np.linspace(1, -1, n)).astype(F)
    x = g.normal(size=n).astype(F)
    yield x
    x = x.copy()
    x[300] = size                                                                    # one, late
    yield x
    x = (x - F(size)).astype(F)                                                      # far below, then near zero
    x[200:] = g.normal(size=n - 200)
    yield x
    x = (size * g.uniform(0.5, 1, n)).astype(F)                                      # none in the first tiles, and one among others
    x[:g.integers(129, 300)] = x[390] = -math.inf
    yield x


SIZES = [2.0 ** e for e in (0, 6, 10, 16, 19, 19.99, 20, 20.01, 21, 24, 26, 27, 28, 29, 30, 33, 36, 39, 40, 41, 50, 51, 52, 60, 100)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("scale", [1.0, -1.0, 0.0883883461356163])
@pytest.mark.parametrize("size", SIZES)
def test_weights_are_held_and_right(size, scale, kind):
    for seed in range(8):
        for scores in cases(size, seed):
            weights, total, (m, lo), most = row(scores if scale > 0 else -scores, scale, kind)
            assert most <= 2
            up, limit = TYPES[kind]
            assert (2.0 ** (up - 0.1) if size < 2.0 ** 36 else min(1, 2.0 ** up)) <= weights.max() <= max(limit, 1)
            f = np.float64(F(scale * 1.4426950408889634))
            x = scores.astype(np.float64) * (f if f > 0 else -f)
            want = np.exp2(x - x.max())
            want /= want.sum()
            # exponents are off by half a last place of numbers up to 126, three times (2^-16), and of the offset's rest; where
            # that is above 2^9, neighbouring scores lie more than 126 apart, and all exponents that count have the same error
            # (below: half a last place of 2^9, 2^-15), of no more than 2^-9, which the logarithm has.  Weights and sums: 2^-21
            # exponentials below 2^-126 are 0
            off = np.abs(weights.astype(np.float64) / total - want)
            assert (off <= want * 2.0 ** -13 + 2.0 ** (-125 - min(0, up))).all(), (off / np.maximum(want, 1e-30)).max()
            lse = np.float64(m) + (np.float64(lo) + math.log2(total))
            exact = x.max() + math.log2(np.exp2(x - x.max()).sum())
            assert abs(lse - exact) <= 2.0 ** -8 + 2.0 ** -40 * abs(exact)


def test_one_number_does_not_do():
    """An offset of one number stays too low for good, from scores of about 2^24 on."""
    never = {e: sum(row(np.full(256, F(2.0 ** e * u)), 1.0, "f16", two=False) is None for u in np.random.default_rng(e).uniform(0.5, 1, 200))
             for e in (18, 20, 25, 29, 32, 36)}
    assert never[18] == never[20] == 0
    assert never[25] > 10 and never[29] > 50 and never[32] > 50 and never[36] > 50
