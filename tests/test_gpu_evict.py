"""GPU parity of the slots' attention weights (within counted roundings) and of the eviction (bit for bit) against plain
restatements."""
import math

import pytest
import torch

import cache_reference as cref
import prompt_reference as ref
from sampling_row_online_gb300 import binding
from test_gpu_cache import ints, make_cache, on_gpu, same_state

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


# ---------------------------------------------------------------- weights
def weigh(kind, dtype, B, N, Hq, Hk, D, page, ctx, counts=None, mask=None, scale=None, seed=0, q=None, dead=()):
    """Runs the call after the attention and checks it; returns the new weights."""
    most = max(c + N for c in ctx)
    state = make_cache(B, most, Hk, page, D, kind, seed)
    cache, table = on_gpu(state)
    host = cref.Cache(*state, kind)
    g = torch.Generator().manual_seed(seed + 1)
    if q is None:
        q = torch.randn((B, N, Hq, D), generator=g).to(dtype).cuda()
    cnt = counts or [N] * B
    on = None if counts is None else ints(*counts)
    words = None if mask is None else mask_words(mask).cuda()
    _, lse = binding.spec_cache_attention(q, cache, table, ints(*ctx), counts=on, mask=words, scale=scale, want_lse=True)
    for b, i, h in dead:
        lse[b, i, h] = -math.inf
    old = torch.rand((B, Hk, table.shape[1] * page), generator=g)
    weights = old.cuda()
    binding.spec_cache_weights(q, cache, table, ints(*ctx), lse, weights, counts=on, mask=words, scale=scale)
    assert binding.spec_get_status() == 0
    got = weights.cpu()
    for b in range(B):
        n = ctx[b] + cnt[b]
        assert torch.equal(got[b, :, n:], old[b, :, n:])
        if cnt[b] == 0:
            assert torch.equal(got[b], old[b])
            continue
        want, tol = ref.slot_weights(host, b, ctx[b], cnt[b], q[b].cpu().double(), lse[b].cpu().double(), None if mask is None else mask[b],
                                     D ** -0.5 if scale is None else scale)
        want[:, :ctx[b]] += old[b, :, :ctx[b]]
        off = (got[b, :, :n].double() - want).abs()
        # exponentials below fp32's least normal number are zero, so each row that sees a slot may miss up to 2^-126 of it
        least = cnt[b] * (Hq // Hk) * 2.0 ** -126
        assert (off <= tol + 2.0 ** -23 * want + least).all(), ((off - tol) / want.clamp(min=1e-3)).max().item()
    return got


def mask_words(mask):
    B, N, _ = mask.shape
    W = (N + 31) // 32
    bits = torch.zeros((B, N, W * 32), dtype=torch.int64)
    bits[..., :N] = mask
    words = (bits.reshape(B, N, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("N,Hq,Hk", [(1, 2, 2), (1, 8, 2), (5, 7, 1), (33, 8, 2), (130, 6, 3)])
def test_weights(kind, dtype, D, page, N, Hq, Hk):
    weigh(kind, dtype, 4, N, Hq, Hk, D, page, [0, 1, page, 4 * page + 7], seed=N + D)


def test_weights_counts_and_chunks():
    """Ragged counts, none among them; more rows than are weighed at a time; many sequences."""
    weigh("e4m3", BF16, 5, 40, 8, 2, 64, 32, [5, 0, 70, 200, 31], counts=[40, 0, 1, 17, 39], seed=3)
    weigh("int8", BF16, 2, 300, 4, 1, 128, 64, [100, 700], counts=[300, 123], seed=4)
    weigh("e4m3", F16, 300, 1, 2, 1, 64, 16, [(7 * b) % 150 for b in range(300)], seed=5)


@pytest.mark.parametrize("N", [7, 63])
def test_weights_under_a_mask(N):
    g = torch.Generator().manual_seed(N)
    mask = torch.rand((3, N, N), generator=g) < 0.4
    mask[:, 2] = False                                     # a token that sees the context alone
    weigh("e4m3", BF16, 3, N, 8, 2, 128, 32, [0, 50, 129], mask=mask, seed=6)   # at ctx 0 it sees nothing


def test_weights_of_rows_that_see_nothing_and_scales():
    weigh("e4m3", BF16, 2, 3, 4, 2, 64, 16, [20, 40], seed=7, dead=[(0, 1, 2), (1, 0, 0), (1, 0, 1)])
    for scale in (0.0, -0.2, 1.0):
        weigh("int8", F16, 2, 4, 4, 2, 64, 16, [33, 5], scale=scale, seed=8)


def test_weights_take_any_strides():
    g = torch.Generator().manual_seed(9)
    B, N, Hq, D = 2, 6, 4, 64
    base = torch.randn((B, Hq, N, D + 1), generator=g).to(BF16).cuda()
    weigh("e4m3", BF16, B, N, Hq, 2, D, 16, [30, 61], seed=9, q=base[..., 1:].transpose(1, 2))
    weigh("e4m3", BF16, B, N, Hq, 2, D, 16, [30, 61], seed=9, q=base[..., :D].transpose(1, 2))


def test_weights_of_bad_pages_and_slots():
    B, N, Hq, Hk, D, page = 3, 2, 4, 2, 64, 16
    state = make_cache(B, 100, Hk, page, D, "e4m3", 10)
    cache, table = on_gpu(state)
    q = torch.randn((B, N, Hq, D), device="cuda").to(BF16)
    ctx = ints(90, 50, 50)
    _, lse = binding.spec_cache_attention(q, cache, table, ctx, want_lse=True)
    old = torch.rand((B, Hk, table.shape[1] * page), device="cuda")
    want = old.clone()
    binding.spec_cache_weights(q, cache, table, ctx, lse, want)
    assert binding.spec_get_status() == 0
    bad = table.clone()
    bad[0, 2] = cache.k.shape[0]
    bad[1, 0] = -1
    got = old.clone()
    binding.spec_cache_weights(q, cache, bad, ctx, lse, got)
    assert binding.spec_get_status() == 9
    want[0, :, 32:48], want[1, :, :16] = old[0, :, 32:48], old[1, :, :16]
    assert torch.equal(got, want)
    got = old.clone()
    binding.spec_cache_weights(q, cache, table, ints(90, table.shape[1] * page, -1), lse, got)
    assert binding.spec_get_status() == 1
    assert torch.equal(got[1:], old[1:]) and torch.equal(got[0, :, :32], want[0, :, :32])


@pytest.mark.parametrize("kind,dtype", [("e4m3", BF16), ("int8", F16)])
@pytest.mark.parametrize("low,high", [(-8, 6), (-9, 6), (-40, 3), (0, 0)])
def test_weights_of_queries_far_apart(kind, dtype, low, high):
    """Rows whose largest elements lie 2^14, 2^15 and more apart, one of zeros among them: a power of two for all or for each."""
    g = torch.Generator().manual_seed(13)
    B, N, Hq, D = 2, 33, 8, 128
    q = torch.randn((B, N, Hq, D), generator=g).clamp(-1.9, 1.9)
    q[..., 0] = 1.5
    low = max(low, -13) if dtype == F16 else low               # fp16's least normal number
    power = torch.randint(low, high + 1, (B, N, Hq, 1), generator=g)
    power[0, 0, :4], power[0, 32, 4:] = low, high
    power[1] = power[0]
    q = q * 2.0 ** power
    q[0, 5, 3] = 0
    weigh(kind, dtype, B, N, Hq, 2, D, 64, [200, 3], seed=13, q=q.to(dtype).cuda())


def test_weights_under_a_mask_of_several_chunks():
    g = torch.Generator().manual_seed(70)
    mask = torch.rand((3, 70, 70), generator=g) < 0.5
    mask[:, torch.arange(70), torch.arange(70)] = True
    weigh("e4m3", BF16, 3, 70, 8, 2, 128, 32, [0, 90, 129], mask=mask, seed=14)
    weigh("int8", F16, 3, 70, 14, 2, 64, 16, [64, 1, 200], mask=mask, counts=[70, 33, 5], seed=15)


# ---------------------------------------------------------------- eviction
def evict(kind, B, Hk, D, page, ctx, keep, first, last, seed=0, weights=None):
    state = make_cache(B, max(ctx), Hk, page, D, kind, seed)
    cache, table = on_gpu(state)
    want = cref.Cache(*state, kind)
    S = table.shape[1] * page
    g = torch.Generator().manual_seed(seed + 2)
    if weights is None:
        weights = torch.randn((B, Hk, S), generator=g).mul(3).exp()
        weights[torch.rand((B, Hk, S), generator=g) < 0.2] = 0   # ties
    on = weights.cuda()
    index, left = binding.spec_cache_evict(cache, table, ints(*ctx), on, keep, first=first, last=last)
    assert binding.spec_get_status() == 0
    new = weights.clone()
    for b in range(B):
        assert int(left[b]) == min(ctx[b], keep)
        rows = [want.rows(t, b, 0, ctx[b]) for t in (0, 1)]
        moved = [[], []]
        for h in range(Hk):
            kept = ref.keeps(weights[b, h].tolist(), ctx[b], keep, first, last)
            assert index[b, h].tolist() == kept + [-1] * (keep - len(kept)), (b, h)
            if ctx[b] > keep:
                new[b, h, :keep] = weights[b, h][kept]
            for t in (0, 1):
                moved[t].append(rows[t][kept, h])
        if ctx[b] > keep:
            for t in (0, 1):
                want.put(t, b, 0, torch.stack(moved[t], 1), True)
    assert torch.equal(on.cpu().nan_to_num(-7.0), new.nan_to_num(-7.0))
    same_state(cache, want)
    return cache, table


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (128, 64), (64, 128)])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (17, 3, 5), (64, 0, 0), (100, 4, 32), (100, 60, 40), (129, 0, 129)])
def test_evict(kind, D, page, keep, first, last):
    evict(kind, 5, 3, D, page, [keep, keep + 1, max(keep - 1, 0), 2 * keep + 37, 400], keep, first, last, seed=keep + D)


def test_evict_many_slots_and_blocks():
    evict("e4m3", 2, 2, 64, 16, [9001, 5000], 2500, 4, 100, seed=1)       # several stretches of rows
    evict("int8", 1, 1, 128, 128, [6000], 1500, 0, 0, seed=2)
    evict("e4m3", 40, 1, 64, 16, [33 + 7 * b for b in range(40)], 48, 2, 2, seed=3)


def test_evict_more_slots_than_shared_memory_holds():
    """Slots that no cluster holds together, and a short context behind the same wide table."""
    evict("int8", 2, 1, 64, 128, [350001, 600], 20000, 3, 1000, seed=4)
    evict("e4m3", 2, 1, 64, 128, [50003, 49000], 300, 0, 0, seed=5)   # two to four CTAs' slices


def test_evict_orders_any_weights():
    """Infinities, NaN, negative and equal weights, both zeros, neighbours in the last bit, and numbers whose digits are equal up
    to any of the three histograms."""
    B, Hk, page, ctx = 2, 2, 16, 500
    S = (-(-ctx // page) + 2) * page
    g = torch.Generator().manual_seed(4)
    pool = torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, 3.4e38, 1.0000001, 0.99999994, 2.0, -2.0])
    w = pool[torch.randint(0, len(pool), (B, Hk, S), generator=g)]
    for keep in (1, 37, 250, 499):
        evict("e4m3", B, Hk, 64, page, [ctx, ctx], keep, 0, 0, seed=5, weights=w)
    near = (torch.full((B, Hk, S), 1.0).view(torch.int32) + torch.randint(0, 5000, (B, Hk, S), generator=g, dtype=torch.int32)).view(torch.float32)
    for keep in (3, 201):
        evict("int8", B, Hk, 64, page, [ctx, 333], keep, 1, 1, seed=6, weights=near)
    evict("int8", B, Hk, 64, page, [ctx, 333], 100, 1, 1, seed=6, weights=torch.zeros(B, Hk, S))


def test_evict_twice_and_foreign_scales():
    """What has been evicted is a cache like any other; scales that are not powers of two are rounded once."""
    state = make_cache(1, 300, 2, 16, 64, "e4m3", 7)
    state = (state[0], state[1], state[2] * 1.3, state[3] * 0.7, state[4])
    cache, table = on_gpu(state)
    want = cref.Cache(*state, "e4m3")
    w = torch.rand((1, 2, table.shape[1] * 16), generator=torch.Generator().manual_seed(1))
    on, ctx = w.cuda(), ints(300)
    for n, keep in ((300, 200), (200, 64)):
        index, ctx = binding.spec_cache_evict(cache, table, ctx, on, keep, first=2, last=10)
        new = w.clone()
        for t in (0, 1):
            # products of codes and scales are rounded to 32 bits, as are their quotients
            full = torch.stack([want.row_f32(t, 0, s) for s in range(n)])
            rows = torch.stack([full[ref.keeps(w[0, h].tolist(), n, keep, 2, 10), h] for h in range(2)], 1)
            for at in range(0, keep, 16):
                p = int(table[0, at // 16])
                for h in range(2):
                    x = rows[at:at + 16, h]
                    scale = cref.scale_for(x.abs().max().item(), "e4m3")
                    want.scales[t][p, h] = scale
                    want.codes[t][p, h].view(torch.uint8)[:len(x)] = cref.nearest((x / scale).double(), "e4m3").view(torch.uint8)
        for h in range(2):
            new[0, h, :keep] = w[0, h][ref.keeps(w[0, h].tolist(), n, keep, 2, 10)]
        w = new
        assert index.shape == (1, 2, keep) and torch.equal(on.cpu(), w)
        same_state(cache, want)
    assert binding.spec_get_status() == 0


def test_evict_leaves_what_it_cannot_move():
    state = make_cache(4, 100, 2, 16, 64, "int8", 8)
    cache, table = on_gpu(state)
    table[1, 3] = cache.k.shape[0]
    table[3, 5] = -1
    S = table.shape[1] * 16
    w = torch.rand((4, 2, S), device="cuda")
    before = [x.clone() for x in (w, cache.k, cache.v, cache.k_scale, cache.v_scale)]
    ctx = ints(S + 1, 100, -1, 40)
    index, left = binding.spec_cache_evict(cache, table, ctx, w, 40)
    assert binding.spec_get_status() in (1, 9)
    assert left.tolist() == ctx.tolist()
    assert (index[:3] == -1).all()
    assert index[3, 0].tolist() == list(range(40))          # nothing to move: its bad page is not looked at
    for a, x in zip(before, (w, cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a.view(torch.uint8), x.view(torch.uint8))
    binding.spec_get_status()


def test_attention_after_eviction_of_idle_slots():
    """Slots that received nothing can go: the attention over what is left is the attention over all."""
    B, Hk, G, D, page, ctx = 2, 2, 4, 64, 16, 200
    cache, table = on_gpu(make_cache(B, ctx + 1, Hk, page, D, "e4m3", 9, spread=0))
    g = torch.Generator().manual_seed(2)
    keys = torch.randn((B, ctx, Hk, D), generator=g) * 0.1
    keys[..., 0] = -40.0
    busy = torch.rand((B, ctx, Hk), generator=g) < 0.25
    keys[..., 0] += 40.0 * busy
    values = torch.randn((B, ctx, Hk, D), generator=g)
    binding.spec_cache_write(cache, table, ints(0, 0), keys.to(BF16).cuda(), values.to(BF16).cuda())
    q = torch.randn((B, 1, Hk * G, D), generator=g)
    q[..., 0] = 30.0
    q = q.to(BF16).cuda()
    new = torch.randn((B, 1, Hk, D), generator=g)
    new[..., 0] = 0
    new = new.to(BF16).cuda()
    lens = ints(ctx, ctx)
    binding.spec_cache_write(cache, table, lens, new, new)
    out, lse = binding.spec_cache_attention(q, cache, table, lens, want_lse=True)
    w = torch.zeros((B, Hk, table.shape[1] * page), device="cuda")
    binding.spec_cache_weights(q, cache, table, lens, lse, w)
    keep = int(busy.sum(1).max()) + 9
    index, left = binding.spec_cache_evict(cache, table, lens, w, keep, last=8)
    for b in range(B):
        for h in range(Hk):
            assert set(busy[b, :, h].nonzero()[:, 0].tolist()) <= set(index[b, h].tolist())
    binding.spec_cache_write(cache, table, left, new, new)
    again, _ = binding.spec_cache_attention(q, cache, table, left)
    assert binding.spec_get_status() == 0
    # codes may be rounded once more where a block's scale differs: keys by half a step of e4m3 (2^-4) of 0.1 to 0.5 in 63
    # places, scores by up to 0.5 * 2^-4 * sum |q| / 8 < 0.3, values by 2^-4
    assert (again.float() - out.float()).abs().max() < 0.6 * values.abs().max()


def test_captured():
    """Weights and eviction in a graph, replayed, give what eager calls give."""
    B, N, Hq, Hk, D, page, ctx = 3, 4, 8, 2, 128, 32, 300
    state = make_cache(B, ctx + N, Hk, page, D, "e4m3", 11)
    q = torch.randn((B, N, Hq, D), device="cuda").to(BF16)
    lens = ints(ctx, ctx - 100, 90)
    caches = [on_gpu(state) for _ in range(3)]
    lse = binding.spec_cache_attention(q, caches[0][0], caches[0][1], lens, want_lse=True)[1]
    w = [torch.zeros((B, Hk, caches[0][1].shape[1] * page), device="cuda") for _ in range(3)]

    def step(i):
        binding.spec_cache_weights(q, caches[i][0], caches[i][1], lens, lse, w[i])
        return binding.spec_cache_evict(caches[i][0], caches[i][1], lens, w[i], 128, first=2, last=16)

    eager = step(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = step(2)
        graph.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(w[i], w[0]) and torch.equal(caches[i][0].k.view(torch.uint8), caches[0][0].k.view(torch.uint8))
        assert torch.equal(caches[i][0].v_scale, caches[0][0].v_scale)
    assert torch.equal(captured[0], eager[0]) and torch.equal(captured[1], eager[1])
    assert binding.spec_get_status() == 0 and binding.spec_get_status(side) == 0
