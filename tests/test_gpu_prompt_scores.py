"""The attention over whole prompts at scores of any size, against a plain 64-bit restatement.  Scores are two products of
short numbers, or one, and nearly all of them exact 32-bit numbers, so that the softmax of scores far apart is well defined."""
import math

import pytest
import torch

from cache_reference import HALF_STEP
from sampling_row_online_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def inputs(T, Hq, Hk, D, dtype, seed):
    """q and k of zeros but for two columns, values as usual: scores are 2^8 k[..., 0] + k[..., 1]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = torch.zeros((T, Hq, D), device="cuda"), torch.zeros((T, Hk, D), device="cuda")
    q[..., 0], q[..., 1] = 256, 1
    v = torch.randn((T, Hk, D), generator=g, device="cuda")
    u = torch.rand((T, Hk), generator=g, device="cuda")
    few = (torch.randn((T, Hk), generator=g, device="cuda") * 8).round() / 8  # eighths
    return q.to(dtype), k, v.to(dtype), u, few


def column(kind, T, u, few):
    """(k[..., 0], k[..., 1]): scores of up to 2^15, in eighths at the finest."""
    zero = torch.zeros_like(u)
    short = lambda x: (x * 128).round()  # noqa: E731  seven bits
    if kind == "alike":
        return zero + 128, zero
    if kind == "different":
        return short((1 + u) / 2), zero
    if kind == "near":                       # alike but for a few units
        return zero + 128, few
    if kind == "negative":
        return -short((1 + u) / 2), few
    ramp = torch.linspace(-1, 1, T, device="cuda")[:, None].expand_as(u)
    if kind == "rising":
        return short(ramp), zero
    if kind == "falling":
        return -short(ramp), few
    late = zero.clone()
    late[T * 3 // 4] = 128
    if kind == "late":
        return late, few
    assert kind == "below"                   # far below, then near zero
    low = zero.clone()
    low[:T // 2] = -128
    return low, few


def check(q, k, v, starts, scale, first=0):
    """first: a sequence's first row that is compared."""
    on = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out, lse = binding.spec_prompt_attention(q, k, v, on, scale=scale, want_lse=True)
    assert binding.spec_get_status() == 0
    G, half = q.shape[1] // k.shape[1], HALF_STEP[q.dtype]
    for lo, hi in zip(starts, starts[1:]):
        later = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device="cuda").triu(1)
        for h in range(q.shape[1]):
            products = q[lo:hi, h].double() @ k[lo:hi, h // G].double().T
            s = (products * scale).masked_fill(later, -math.inf)
            z, vv = torch.logsumexp(s, -1), v[lo:hi, h // G].double()
            top = s.amax(-1, keepdim=True)
            w = (s - top).exp()
            w /= w.sum(-1, keepdim=True)
            want, spread = w @ vv, w @ vv.abs()
            # exponents: half a last place of numbers up to 126, three times (2^-16); an offset's, which is the same for all
            # weights of a row; and that of a large offset's rest (below 2^9: 2^-15; above, scores that differ lie more than
            # 126 apart).  The exponential and the sums: 2^-20.  So a weight is off by less than 2^-14 of it, and so is their
            # sum
            tol = (half + 2.0 ** -13) * spread
            # a score that 32 bits do not hold is off by a last place at most (one addition, rounded or cut off), so a weight
            # by a factor of e to that, and so is their sum
            seen = products[s.isfinite()]
            place = 0.0 if torch.equal(seen.float().double(), seen) else 2.0 ** -23 * seen.abs().max().item() * abs(scale)
            tol += math.expm1(2 * place) * spread
            if q.dtype == F16:  # fp16's least step, half of which is 2^-25 where the largest weight is 2^7.9 (1 beyond 2^40)
                least = 2.0 ** -25 if abs(scale) >= 2.0 ** 24 else 2.0 ** -32
                tol += least * w.amax(-1, keepdim=True) * ((~later).double() @ vv.abs())
            off = (out[lo:hi, h].double() - want).abs()
            assert (off <= tol + half * want.abs() * 1.01 + half * tol)[first:].all(), (h, off.max().item())
            # the logarithm: the factor of the scores, the offset, its product with ln 2, each to half a last place
            off = (lse[lo:hi, h].double() - z).abs()
            assert (off <= 2.0 ** -13 + 2.0 ** -22 * z.abs() + place)[first:].all(), (h, off.max().item())


KINDS = ["alike", "different", "near", "negative", "rising", "falling", "late", "below"]


@pytest.mark.parametrize("power", [0, 6, 10, 14, 18, 30])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_any_size(D, dtype, kind, power):
    """Scores of up to 2^15 times 2^power, of both signs."""
    T = 700
    q, k, v, u, few = inputs(T, 4, 2, D, dtype, power)
    k[..., 0], k[..., 1] = column(kind, T, u, few)
    k = k.to(dtype)
    check(q, k, v, [0, 90, 700], 2.0 ** power)
    check(q, k, v, [0, 90, 700], -2.0 ** power)


@pytest.mark.parametrize("power", [6, 14, 30])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,D,dtype", [(2, 128, BF16), (2, 64, F16), (3, 128, F16)])
def test_scores_of_any_size_over_many_ctas(Hq, D, dtype, kind, power):
    """One sequence whose pieces are joined."""
    T = 4500
    q, k, v, u, few = inputs(T, Hq, 1, D, dtype, power)
    k[..., 0], k[..., 1] = column(kind, T, u, few)
    check(q, k.to(dtype), v, [0, T], 2.0 ** power)


@pytest.mark.parametrize("D", [64, 128])
def test_large_elements(D):
    """The size lies in the elements, not in the scale: fp16's largest, and bf16's up to products near 2^120."""
    T = 300
    for dtype, a, b in ((F16, 65504.0, 65504.0), (BF16, 2.0 ** 60, 2.0 ** 60), (BF16, 1e20, 1e10)):
        q, k, v, u, _ = inputs(T, 4, 2, D, dtype, 3)
        q[..., 0], q[..., 1] = a, 0
        k[..., 0] = b * u
        check(q, k.to(dtype), v, [0, T], D ** -0.5)
        k[..., 0] = b
        check(q, k.to(dtype), v, [0, T], D ** -0.5)


@pytest.mark.parametrize("rest", ["near zero", "far below", "beyond", "whole"])
@pytest.mark.parametrize("keys", [(0, 127), (0, 128), (0, 300), (256, 384), (130, 690)], ids=str)
@pytest.mark.parametrize("Hq,Hk,D,dtype,T", [(4, 2, 128, BF16, 700), (4, 2, 64, F16, 700), (6, 2, 128, F16, 700), (2, 1, 128, BF16, 4500),
                                             (3, 1, 64, F16, 4500)])
def test_keys_that_count_nothing(Hq, Hk, D, dtype, T, keys, rest):
    """Some keys' scores are -inf, by an infinite element: a row's softmax is that over the others, wherever they stand."""
    q, k, v, u, few = inputs(T, Hq, Hk, D, dtype, keys[1])
    k[..., 1] = few
    if rest == "far below":
        k[..., 0] = -1                       # scores of -256
    if rest == "beyond":
        k[..., 0] = -2.0 ** 15               # of -2^23 and some eighths, which 32 bits do not hold
    if rest == "whole":
        k[..., 0], k[..., 1] = -2.0 ** 14, few.round()
    q[..., 2] = 1
    lo, hi = (x * T // 700 for x in keys)
    k[lo:hi, :, 2] = -math.inf
    q, k = q.to(dtype), k.to(dtype)
    if lo == 0:                              # rows that see no other key have no softmax
        on = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        out, lse = binding.spec_prompt_attention(q, k, v, on, scale=1.0, want_lse=True)
        assert out[:hi].isnan().all() and not lse[:hi].isfinite().any()
    check(q, k, v, [0, T], 1.0, hi if lo == 0 else 0)


@pytest.mark.parametrize("size", [1e-25, 1e30, 1e36, 3.3895313892515355e38])
@pytest.mark.parametrize("Hq,Hk,D,T", [(4, 2, 64, 700), (4, 2, 128, 700), (2, 1, 128, 4500), (3, 1, 64, 4500)])
def test_values_of_any_size(Hq, Hk, D, T, size):
    """An average of bf16 values is finite, however large they are: up to the type's largest."""
    q, k, v, u, few = inputs(T, Hq, Hk, D, BF16, 4)
    for scores in (0 * few, few):
        k[..., 1] = scores
        sign = torch.where(torch.rand(v.shape, device="cuda") < 0.9, 1.0, -1.0)
        check(q, k.to(BF16), (sign * size).to(BF16), [0, 100, T], 1.0)
        check(q, k.to(BF16), torch.full_like(v, size), [0, T], 1.0)


@pytest.mark.parametrize("junk", [30.0, 2.0 ** 14, -2.0 ** 14, math.inf, math.nan])
@pytest.mark.parametrize("Hq,Hk,D,dtype,T", [(4, 1, 128, BF16, 700), (4, 1, 64, F16, 700), (6, 2, 64, BF16, 700), (2, 1, 128, F16, 4500)])
def test_later_queries_change_nothing(Hq, Hk, D, dtype, T, junk):
    """A row's result, to the last bit, is its own: whatever the queries, keys and values of later rows are."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda").to(dtype) for H in (Hq, Hk, Hk))
    on = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    clean = binding.spec_prompt_attention(q, k, v, on, want_lse=True)
    for t in (1, 130, 277, T - 3):
        for which in ((0,), (0, 1, 2)):
            x = [y.clone() for y in (q, k, v)]
            for i in which:
                x[i][t:] = x[i][t:] * junk if i == 0 and math.isfinite(junk) else junk
            out, lse = binding.spec_prompt_attention(*x, on, want_lse=True)
            assert torch.equal(out[:t], clean[0][:t]) and torch.equal(lse[:t], clean[1][:t])
    assert binding.spec_get_status() == 0
