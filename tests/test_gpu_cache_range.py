"""The attention at the ends of its range: value scales near the least that counts and far from one another, many tiles
of tokens, and many new tokens."""
import math

import pytest
import torch

import cache_reference as ref
from sampling_row_online_gb300 import SpecCache, binding
from test_gpu_cache import BF16, F16, ints, make_cache, mask_of, on_gpu, random_trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("N", [1, 30])
@pytest.mark.parametrize("power", [-100, -99, -80, 0, 118])
@pytest.mark.parametrize("slots", [31, 2000, 2 ** 17 + 40])
@pytest.mark.parametrize("rise", [0.0, 2.75, 7.5])
def test_equal_values_under_scales_of_any_size(kind, D, N, power, slots, rise):
    """One sequence whose values are equal: out is that value, and the softmax's sum n0 + n1 2^rise, with n0 = 128 slots
    (or all) of score 0 and then n1 of a score that lets weights rise as far as they may before the offset moves."""
    page = 64
    pages = -(-slots // page)
    k = torch.ones((pages, 1, page, D), device="cuda")
    k[:2] = 0
    v = torch.full((pages, 1, page, D), 3.0, device="cuda")
    k, v = (t.to(ref.CODE[kind]) for t in (k, v))
    cache = SpecCache(k, v, torch.full((pages, 1), rise * math.log(2), device="cuda"), torch.full((pages, 1), 2.0 ** power, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = torch.ones((1, N, 2, D), dtype=BF16, device="cuda")
    ctx = slots - N
    out, lse = binding.spec_cache_attention(q, cache, table, ints(ctx), scale=1 / D, want_lse=True)
    assert binding.spec_get_status() == 0
    value = 3.0 * 2.0 ** power if power > -100 else 0.0   # scales up to 2^-100 count as 0
    # weights' rounding to fp16, the output's to bf16; the sum and the products over up to 2^17 slots are sums of pieces of
    # some thousands in 32 bits
    assert bool(((out.double() - value).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -10) * value).all())
    n = ctx + 1 + torch.arange(N, device="cuda").double()
    want = (n.clamp(max=128) + (n - 128).clamp(min=0) * 2.0 ** rise).log()[None, :, None]
    assert bool(((lse.double() - want).abs() <= 2.0 ** -10).all())


def wide_reference(cache, b, ctx, cnt, q, mask, scale):
    """ref.attention with the least step of weights whose largest is at least 2^8 (eight or more tiles of 128 tokens in the
    tile kernel): half of fp16's 2^-24 is 2^-33 of it, once per slot."""
    out, lse, to, tl = ref.attention(cache, b, ctx, cnt, q, mask, scale)
    N, Hq, D = q.shape
    k, (codes, vs) = cache.rows(0, b, 0, ctx + cnt), cache.rows(1, b, 0, ctx + cnt, scaled=False)
    group = Hq // k.shape[1]
    seen = torch.zeros((N, ctx + cnt), dtype=torch.bool)
    seen[:, :ctx] = True
    seen[:, ctx:] = (torch.arange(cnt)[None] <= torch.arange(N)[:, None]) if mask is None else mask[:, :cnt]
    seen[cnt:] = False
    s = torch.einsum("nhd,thd->nht", q, k.repeat_interleave(group, 1)) * scale
    p = torch.where(seen[:, None], (s - lse[..., None].clamp(min=-1e300)).exp(), 0.0)
    top = (p * vs.repeat_interleave(group, 1).T[None]).amax(-1)
    least = 2.0 ** -33 * top[..., None] * torch.einsum("nt,thd->nhd", seen.double(), codes.abs().repeat_interleave(group, 1))
    return out, lse, to + least, tl


def check(state, kind, ctx, q, words, scale=None):
    N, D = q.shape[1], q.shape[3]
    cache, table = on_gpu(state)
    out, lse = binding.spec_cache_attention(q.cuda(), cache, table, ints(*ctx), mask=None if words is None else words.cuda(),
                                            scale=scale, want_lse=True)
    assert binding.spec_get_status() == 0
    out, lse, want = out.cpu().double(), lse.cpu().double(), ref.Cache(*state, kind)
    for b in range(len(ctx)):
        o, l, to, tl = wide_reference(want, b, ctx[b], N, q[b].double(), None if words is None else mask_of(words[b], N),
                                      D ** -0.5 if scale is None else scale)
        tol = to + ref.HALF_STEP[q.dtype] * o.abs() + (2.0 ** -25 if q.dtype == F16 else 1e-30)
        assert torch.all((out[b] - o).abs() <= tol), b
        assert torch.all((lse[b] - l).abs() <= tl), b


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("N,Hq", [(1, 4), (5, 8), (20, 8)])
def test_value_scales_far_apart_over_many_tiles(kind, N, Hq):
    """Value scales that differ by up to 2^79 within a row, some of them zero, over more than eight tiles of tokens."""
    state = make_cache(2, 1500 + N, 2, 16, 64, kind, 6, spread=0)
    g = torch.Generator().manual_seed(4)
    ks, vs = state[2], state[3]
    ks.mul_(torch.rand(ks.shape, generator=g) + 0.5)
    q = torch.randn((2, N, Hq, 64), generator=g).to(BF16)
    for powers in (torch.rand(vs.shape, generator=g) * 79 - 60, (torch.rand(vs.shape, generator=g) < 0.1) * 79.0 - 60):
        vs.copy_(torch.exp2(powers))
        vs[::5] = 0
        check(state, kind, [1500, 1100], q, None)
        check(state, kind, [1500, 1100], q * 30, None)                   # a few slots carry each row


@pytest.mark.parametrize("kind,D,dtype", [("e4m3", 128, BF16), ("int8", 64, F16)])
@pytest.mark.parametrize("N,Hq,Hk,ctx", [(1024, 4, 2, [0, 700]), (1500, 2, 2, [37, 1]), (2051, 3, 1, [0, 260])])
def test_many_new_tokens(kind, D, dtype, N, Hq, Hk, ctx):
    """A part of a prompt: every row tile ends at its own last token."""
    state = make_cache(len(ctx), max(ctx) + N, Hk, 64, D, kind, N)
    q = torch.randn((len(ctx), N, Hq, D), generator=torch.Generator().manual_seed(N)).to(dtype)
    check(state, kind, ctx, q, None)


def test_many_new_tokens_under_a_mask():
    N, ctx = 1025, [300, 0]
    g = torch.Generator().manual_seed(3)
    at = torch.arange(N)
    words = torch.zeros((2, N, (N + 31) // 32 * 32), dtype=torch.int64)
    words[..., :N] = (torch.rand((2, N, N), generator=g) < 0.02) | (at[None, :, None] == at[None, None])
    words = (words.reshape(2, N, -1, 32) << torch.arange(32)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    state = make_cache(2, 300 + N, 2, 32, 128, "e4m3", 3)
    check(state, "e4m3", ctx, torch.randn((2, N, 4, 128), generator=g).to(BF16), words)
