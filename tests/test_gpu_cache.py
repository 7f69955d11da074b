"""GPU parity of the operators around the 8-bit paged key/value cache against plain 64-bit restatements: the write and
the commit bit for bit, the others within counted roundings."""
import math

import pytest
import torch

import cache_reference as ref
from sampling_row_online_gb300 import SpecCache, binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make_cache(B, slots, Hk, page, D, kind, seed, spread=2, garbage=True):
    """A pool with a few pages more than are used, a mixed-up table with -1 where nothing is needed for `slots`
    tokens, normal values with scales that differ by up to 2^spread."""
    g = torch.Generator().manual_seed(seed)
    per = -(-slots // page) + 2
    need = -(-slots // page)
    pages = B * need + 3
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, per), -1, dtype=torch.int32)
    table[:, :need] = order[:B * need].reshape(B, need).to(torch.int32)
    codes = []
    for _ in range(2):
        x = torch.randn((pages, Hk, page, D), generator=g) * ref.QMAX[kind] / 4
        x = x.clamp(-ref.QMAX[kind], ref.QMAX[kind])
        codes.append(x.round().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn))
    scales = [torch.ldexp(torch.ones(pages, Hk), torch.randint(-spread, spread + 1, (pages, Hk), generator=g) - (7 if kind == "e4m3" else 5))
              for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1], table


def on_gpu(state):
    k, v, ks, vs, table = state
    return SpecCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda()), table.cuda()


def same_state(cache, want):
    for t, (codes, scales) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert torch.equal(scales.cpu(), want.scales[t])
        got, exp = codes.cpu().view(torch.uint8), want.codes[t].view(torch.uint8)
        if want.kind == "e4m3":  # both zeros are zero
            got, exp = (torch.where(x == 128, 0, x) for x in (got, exp))
        assert torch.equal(got, exp)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,page,D", [(1, 16, 64), (1, 128, 128), (7, 32, 128), (64, 64, 64), (129, 64, 128), (300, 128, 128)])
def test_write(kind, dtype, N, page, D):
    B, Hk = 6, 3
    state = make_cache(B, 2 * page + N + 5, Hk, page, D, kind, N + page)
    g = torch.Generator().manual_seed(N)
    ctx = [0, 1, page - 1, page, page + 3, 2 * page]
    counts = [N, N, max(N - 1, 0), 0, N, (N + 1) // 2]
    # magnitudes that make some blocks grow and leave others
    k, v = (torch.randn((B, N, Hk, D), generator=g) * torch.tensor([1e-3, 1., 30.])[:, None] for _ in range(2))
    k[0, :, 0] = 0
    k, v = k.to(dtype), v.to(dtype)
    want = ref.Cache(*state, kind)
    for b in range(B):
        want.put(0, b, ctx[b], k[b, :counts[b]].double(), True)
        want.put(1, b, ctx[b], v[b, :counts[b]].double(), True)
    cache, table = on_gpu(state)
    binding.spec_cache_write(cache, table, ints(*ctx), k.cuda(), v.cuda(), counts=ints(*counts))
    assert binding.spec_get_status() == 0
    same_state(cache, want)


@pytest.mark.parametrize("layout", ["heads_first", "odd_offset", "broadcast", "backwards_batch"])
def test_write_takes_any_strides(layout):
    B, N, Hk, D, page = 2, 37, 4, 64, 32
    state = make_cache(B, 80, Hk, page, D, "e4m3", 3)
    g = torch.Generator().manual_seed(5)
    if layout == "heads_first":
        k, v = (torch.randn((B, Hk, N, D), generator=g).to(BF16).cuda().transpose(1, 2) for _ in range(2))
    elif layout == "odd_offset":
        k, v = (torch.randn((B, N, Hk, D + 1), generator=g).to(BF16).cuda()[..., 1:] for _ in range(2))
    elif layout == "broadcast":
        k, v = (torch.randn((B, N, 1, D), generator=g).to(BF16).cuda().expand(B, N, Hk, D) for _ in range(2))
    else:
        k, v = (torch.randn((2 * B, N, Hk, D), generator=g).to(BF16).cuda()[::2] for _ in range(2))
    want = ref.Cache(*state, "e4m3")
    for b in range(B):
        want.put(0, b, 20, k[b].cpu().double(), True)
        want.put(1, b, 20, v[b].cpu().double(), True)
    cache, table = on_gpu(state)
    binding.spec_cache_write(cache, table, ints(20, 20), k, v)
    assert binding.spec_get_status() == 0
    same_state(cache, want)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_write_of_extremes(kind):
    """Values at the codes' borders, subnormals of the codes, the least scale, and non-finite ones."""
    page, D = 16, 64
    state = make_cache(1, 64, 1, page, D, kind, 1)
    q = ref.QMAX[kind]
    k = torch.zeros((1, 48, 1, D))
    k[0, 0, 0, :6] = torch.tensor([q, -q, q / 2 + 0.5, 0.5, 1.5, 2.5])             # exactly at the border
    k[0, 16, 0, :5] = torch.tensor([q * 1.0001, q, 1.0, 2.0 ** -10, -2.0 ** -9])  # just over it
    k[0, 32, 0, :2] = torch.tensor([2.0 ** -120, 1e-38])                          # below the least scale
    want = ref.Cache(*state, kind)
    for t in (0, 1):
        want.put(t, 0, 0, k[0].double(), True)
    cache, table = on_gpu(state)
    binding.spec_cache_write(cache, table, ints(0), k.cuda(), k.cuda())
    assert binding.spec_get_status() == 0
    same_state(cache, want)
    k[0, 3, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    for t in (0, 1):
        want.put(t, 0, 0, k[0].double(), True)
    binding.spec_cache_write(cache, table, ints(0), k.cuda(), k.cuda())
    assert binding.spec_get_status() == 10  # SPEC_ERR_NONFINITE
    assert binding.spec_get_status() == 0
    same_state(cache, want)


def test_write_token_by_token_grows_the_scale():
    """A block filled one row at a time ends with the scale of its largest row; e4m3 rows move without a second error."""
    page, D = 64, 128
    state = make_cache(1, page, 2, page, D, "e4m3", 8)
    g = torch.Generator().manual_seed(3)
    k = (torch.randn((1, page, 2, D), generator=g) * torch.linspace(0.1, 40, page)[:, None, None]).to(BF16)
    want = ref.Cache(*state, "e4m3")
    cache, table = on_gpu(state)
    for i in range(page):
        for t in (0, 1):
            want.put(t, 0, i, k[0, i:i + 1].double(), True)
        binding.spec_cache_write(cache, table, ints(i), k[:, i:i + 1].cuda(), k[:, i:i + 1].cuda())
    assert binding.spec_get_status() == 0
    same_state(cache, want)
    got = want.rows(0, 0, 0, page)
    # one rounding of half a step 2^-4, or half the least e4m3 step 2^-9 times the scale (twice: a row may move)
    least = 2 * 2.0 ** -10 * want.scales[0][int(table[0, 0])].double()[None, :, None]
    assert torch.all((got - k[0].double()).abs() <= 2.0 ** -4 * k[0].double().abs() + least)


def test_bad_slots_and_pages_are_reported():
    B, Hk, page, D, N = 3, 2, 16, 64, 8
    state = make_cache(B, 64, Hk, page, D, "e4m3", 4)
    state[4][1, 0] = 10 ** 6                        # sequence 1's first page does not exist
    cache, table = on_gpu(state)
    k = torch.randn((B, N, Hk, D)).to(BF16).cuda()
    ctx = ints(0, 0, 4000)                          # sequence 2 does not fit its pages
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale)]
    binding.spec_cache_write(cache, table, ctx, k, k)
    assert binding.spec_get_status() in (1, 9)
    binding.spec_get_status()
    own = table[0].long().clamp(min=0)
    changed = (cache.k_scale != before[1]).any(1)
    changed[own] = False
    assert not changed.any()                        # only sequence 0 was written
    out, lse = binding.spec_cache_attention(k, cache, table, ctx, want_lse=True)
    assert binding.spec_get_status() in (1, 9)
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(out[1:].float()).all() and torch.isnan(lse[1:]).all()
    rk, rv = binding.spec_cache_read(cache, table, ctx, None, N)
    assert binding.spec_get_status() in (1, 9)
    assert torch.isfinite(rk[0].float()).all() and torch.isnan(rk[1:].float()).all() and torch.isnan(rv[1:].float()).all()


# ------------------------------------------------------------------- read
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,page,D", [(1, 16, 128), (33, 32, 64), (200, 64, 128), (129, 128, 64)])
def test_read(kind, dtype, N, page, D):
    B, Hk = 4, 2
    state = make_cache(B, N + page + 3, Hk, page, D, kind, N)
    start, counts = [0, 1, page - 1, page + 3], [N, N // 2, N, 0]
    cache, table = on_gpu(state)
    got = binding.spec_cache_read(cache, table, ints(*start), ints(*counts), N, dtype=dtype)
    assert binding.spec_get_status() == 0
    want = ref.Cache(*state, kind)
    for t in (0, 1):
        for b in range(B):
            exp = torch.zeros((N, Hk, D), dtype=torch.float64)
            exp[:counts[b]] = want.rows(t, b, start[b], start[b] + counts[b])
            assert torch.equal(got[t][b].cpu(), exp.float().to(dtype))  # powers of two: exact in 32 bits


# -------------------------------------------------------- norms and rotation
def rope_reference(x, w, pos, inv, rot, pairs, norm, eps):
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
    f = pos.double()[..., None] * inv
    c, s = f.cos()[:, :, None], f.sin()[:, :, None]
    out, big = y.clone(), y.abs().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    big[..., a] = big[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, big


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D,rot,pairs,norm", [(128, 128, False, True), (128, 64, True, True), (64, 64, False, False),
                                              (80, 80, False, True), (80, 40, True, True), (256, 256, False, True),
                                              (512, 0, False, True), (96, 18, False, True), (6, 4, True, True), (2, 2, False, True),
                                              (512, 512, False, True)])
@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 1), (3, 7, 8, 2), (2, 700, 3, 1)])
def test_norm_rope(dtype, D, rot, pairs, norm, B, N, Hq, Hk):
    g = torch.Generator().manual_seed(D + N)
    q, k = (torch.randn((B, N, H, D), generator=g).mul(3).to(dtype) for H in (Hq, Hk))
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype) if norm else None for _ in range(2))
    base = torch.randint(0, 2 ** 30, (B,), generator=g, dtype=torch.int32)
    base[0] = 0
    offset = torch.randint(0, 50, (B, N), generator=g, dtype=torch.int32) if N == 7 else None
    pos = base[:, None].long() + (torch.arange(N)[None] if offset is None else offset.long())
    inv = 1e4 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    got = binding.spec_qk_norm_rope(q.cuda(), k.cuda(), inv if rot else None, base=base.cuda(),
                                    offset=None if offset is None else offset.cuda(), norm=norm,
                                    q_weight=None if wq is None else wq.cuda(), k_weight=None if wk is None else wk.cuda(),
                                    eps=1e-5, pairs=pairs)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        exp, big = rope_reference(x, w, pos, inv, rot, pairs, norm, 1e-5)
        # one rounding of the result; in 32 bits a sum of D squares (its root halves that), four products and
        # sums, and an angle of 2^-24 turns; the reference's own angle is off by up to 2^30 2^-53 radians
        tol = ref.HALF_STEP[dtype] * exp.abs() + big * ((D / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) + 1e-30
        if dtype == F16:
            tol = tol + 2.0 ** -25
        assert torch.all((y.cpu().double() - exp).abs() <= tol)


@pytest.mark.parametrize("D,rot,pairs", [(80, 80, False), (128, 48, True), (128, 128, False), (64, 48, False)])
def test_norm_rope_of_many_tokens(D, rot, pairs):
    """Several angles to a thread, whether or not their number divides the threads."""
    test_norm_rope(BF16, D, rot, pairs, True, 3, 5000, 2, 1)


def test_norm_rope_in_place_strided_and_single():
    g = torch.Generator().manual_seed(1)
    both = torch.randn((2, 9, 6, 128), generator=g).to(BF16).cuda()       # q and k heads in one tensor
    q, k = both[:, :, :4], both[:, :, 4:]
    inv = 1e6 ** (-torch.arange(64, dtype=torch.float64) / 64)
    want = binding.spec_qk_norm_rope(q.contiguous(), k.contiguous(), inv)
    only = binding.spec_qk_norm_rope(None, k, inv)
    assert only[0] is None and torch.equal(only[1], want[1])
    odd = torch.empty((2, 9, 4, 129), dtype=BF16, device="cuda")[..., 1:]  # unaligned rows: single elements
    binding.spec_qk_norm_rope(q, None, inv, out_q=odd)
    assert torch.equal(odd, want[0])
    binding.spec_qk_norm_rope(q, k, inv, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


# -------------------------------------------------------------- attention
def random_trees(g, B, N):
    parent = torch.full((B, N), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(1, N):
            parent[b, i] = int(torch.randint(0, i, (1,), generator=g))
    return parent


def mask_of(words, N):
    """[N, W] words as [N, N] bool."""
    bit = (words.long()[..., None] >> torch.arange(32)) & 1
    return bit.reshape(words.shape[0], -1)[:, :N].bool()


def check_attention(state, kind, ctx, counts, q, words, scale=None, run=None):
    B, N, Hq, D = q.shape
    cache, table = on_gpu(state)
    out, lse = (run or binding.spec_cache_attention)(q.cuda(), cache, table, ints(*ctx), counts=None if counts is None else ints(*counts),
                                                     mask=None if words is None else words.cuda(), scale=scale, want_lse=True)
    assert binding.spec_get_status() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    want = ref.Cache(*state, kind)
    for b in range(B):
        cnt = N if counts is None else counts[b]
        o, l, to, tl = ref.attention(want, b, ctx[b], cnt, q[b].double(), None if words is None else mask_of(words[b], N),
                                     D ** -0.5 if scale is None else scale)
        tol = to + ref.HALF_STEP[q.dtype] * o.abs() + (2.0 ** -25 if q.dtype == F16 else 1e-30)
        bad = ~((out[b] - o).abs() <= tol)
        assert not bad.any(), (b, bad.nonzero()[:4].tolist(), (out[b] - o).abs().max().item(), tol.min().item())
        empty = torch.isinf(l)
        assert torch.equal(torch.isneginf(lse[b]), empty)
        assert torch.all(((lse[b] - l).abs() <= tl)[~empty])
    return out, lse


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,D,page", [(BF16, 128, 64), (F16, 128, 16), (BF16, 64, 128), (F16, 64, 32)])
@pytest.mark.parametrize("N,Hq,Hk", [(1, 1, 1), (1, 8, 1), (1, 32, 8), (1, 14, 2), (4, 8, 2), (6, 16, 2), (9, 5, 5), (33, 12, 4)])
def test_attention_of_chains(kind, dtype, D, page, N, Hq, Hk):
    ctx = [0, 1, 15, 16, 17, page, 5 * page + 3, 700]
    state = make_cache(len(ctx), 700 + N, Hk, page, D, kind, N + Hq)
    g = torch.Generator().manual_seed(N * Hq)
    q = torch.randn((len(ctx), N, Hq, D), generator=g).mul(1.5).to(dtype)
    check_attention(state, kind, ctx, None, q, None)


@pytest.mark.parametrize("kind,dtype,D", [("e4m3", BF16, 128), ("int8", F16, 64), ("int8", BF16, 128)])
@pytest.mark.parametrize("N,Hq,Hk", [(2, 4, 2), (31, 4, 4), (63, 8, 2), (65, 3, 1), (130, 4, 2)])
def test_attention_of_trees(kind, dtype, D, N, Hq, Hk):
    g = torch.Generator().manual_seed(N)
    ctx, counts = [0, 3, 200, 333], [N, N - 1, N, 0]
    parent = random_trees(g, 4, N)
    words = binding.spec_tree_mask(parent.cuda())[0].cpu()
    words[1, 1] = 0                                   # a node that sees its context only
    words[0, N // 2] = 0                              # a node that sees nothing
    state = make_cache(4, 333 + N, Hk, 32, D, kind, N)
    q = torch.randn((4, N, Hq, D), generator=g).to(dtype)
    out, lse = check_attention(state, kind, ctx, counts, q, words)
    assert torch.all(out[0, N // 2] == 0) and torch.all(lse[0, N // 2] == -math.inf)
    assert torch.all(out[3] == 0) and torch.all(lse[3] == -math.inf)


@pytest.mark.parametrize("N", [1, 7, 40])
def test_attention_of_long_ragged_contexts(N):
    """Long axes are split over the whole GPU and joined, next to sequences of a few tokens."""
    ctx = [20000, 5, 4097, 0, 1]
    state = make_cache(5, 20000 + N, 2, 64, 128, "e4m3", 9)
    q = torch.randn((5, N, 8, 128), generator=torch.Generator().manual_seed(2)).to(BF16)
    check_attention(state, "e4m3", ctx, None, q, None)


@pytest.mark.parametrize("N", [1, 20])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_attention_scales_of_any_size(kind, N):
    """Scales that are no powers of two, differ by 2^60 between blocks, or are zero; scores that leave one slot."""
    state = make_cache(3, 300 + N, 2, 16, 64, kind, 6, spread=0)
    g = torch.Generator().manual_seed(4)
    ks, vs = state[2], state[3]
    ks.mul_(torch.rand(ks.shape, generator=g) + 0.5)
    vs.mul_(torch.exp(torch.rand(vs.shape, generator=g) * 40 - 20))
    vs[::5] = 0
    ks[::7] = 0
    q = torch.randn((3, N, 4, 64), generator=g).to(BF16)
    check_attention(state, kind, [300, 16, 0], None, q, None)
    check_attention(state, kind, [300, 16, 0], None, q * 100, None)      # nearly one-hot
    check_attention(state, kind, [300, 16, 0], None, q, None, scale=-0.3)
    check_attention(state, kind, [300, 16, 0], None, q, None, scale=0.0)


@pytest.mark.parametrize("N", [1, 30])
def test_attention_ignores_what_is_not_there(N):
    """NaN codes and NaN scales past the last slot, -1 in the table behind it, queries of rows past the count."""
    B, Hk, page, D = 2, 2, 64, 128
    ctx = [70, 5]
    state = make_cache(B, 128 + N, Hk, page, D, "e4m3", 5)
    clean = [t.clone() for t in state]
    for b in range(B):
        last = ctx[b] + N
        for slot in range(last, 128):
            p = int(state[4][b, slot // page])
            for t in (0, 1):
                state[t][p, :, slot % page].view(torch.uint8).fill_(0x7F if slot % 2 else 0xFF)
        for blk in range(-(-last // page), state[4].shape[1]):
            if state[4][b, blk] >= 0:
                state[2][int(state[4][b, blk])] = math.nan
                state[3][int(state[4][b, blk])] = math.inf
            state[4][b, blk] = -1
    q = torch.randn((B, N, 4, D), generator=torch.Generator().manual_seed(3)).to(BF16)
    cache, table = on_gpu(state)
    got = binding.spec_cache_attention(q.cuda(), cache, table, ints(*ctx))[0]
    cache, table = on_gpu(clean)
    want = binding.spec_cache_attention(q.cuda(), cache, table, ints(*ctx))[0]
    assert binding.spec_get_status() == 0
    assert torch.equal(got, want) and torch.isfinite(got.float()).all()


@pytest.mark.parametrize("N", [1, 50])
def test_attention_query_extremes(N):
    """A row of zeros, of large and of tiny values, and one with a NaN, which stays by itself."""
    state = make_cache(1, 200 + N, 1, 32, 64, "int8", 5)
    q = torch.randn((1, N, 8, 64), generator=torch.Generator().manual_seed(3))
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 2.0 ** 20
    q[0, 0, 2] *= 2.0 ** -60
    q = q.to(BF16)
    check_attention(state, "int8", [200], None, q, None, scale=2.0 ** -14)
    bad = q.clone()
    bad[0, 0, 3, 5] = math.nan
    cache, table = on_gpu(state)
    a = binding.spec_cache_attention(q.cuda(), cache, table, ints(200))[0]
    b = binding.spec_cache_attention(bad.cuda(), cache, table, ints(200))[0]
    assert torch.isnan(b[0, 0, 3].float()).all()
    a[0, 0, 3] = 0
    b[0, 0, 3] = 0
    assert torch.equal(a, b)


def test_attention_takes_any_strides():
    state = make_cache(3, 300, 2, 32, 64, "e4m3", 5)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((3, 5, 8, 64), generator=g).to(BF16)
    cache, table = on_gpu(state)
    ctx = ints(290, 17, 0)
    want = binding.spec_cache_attention(q.cuda(), cache, table, ctx)[0]
    other = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(binding.spec_cache_attention(other, cache, table, ctx)[0], want)
    odd = torch.empty((3, 5, 8, 65), dtype=BF16, device="cuda")[..., 1:]
    odd.copy_(q)
    assert torch.equal(binding.spec_cache_attention(odd, cache, table, ctx)[0], want)


@pytest.mark.parametrize("N,Hq", [(1, 8), (20, 8), (70, 16)])
def test_attention_is_deterministic_and_follows_its_stream(N, Hq):
    state = make_cache(7, 3000 + N, 2, 64, 128, "e4m3", 5)
    q = torch.randn((7, N, Hq, 128), generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    cache, table = on_gpu(state)
    ctx = ints(3000, 1, 17, 2048, 999, 0, 64)
    a = binding.spec_cache_attention(q, cache, table, ctx, want_lse=True)
    for _ in range(3):
        b = binding.spec_cache_attention(q, cache, table, ctx, want_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = binding.spec_cache_attention(q, cache, table, ctx, want_lse=True)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_pass_32_bits():
    """A pool of over 2^32 bytes, the sequence's pages at its end."""
    pages, page, D = 300000, 128, 128
    assert pages * page * D > 2 ** 32
    k = torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = SpecCache(k, v, torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"))
    table = torch.tensor([[pages - 1, pages - 3, 7]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    new = torch.randn((1, 300, 1, D), generator=g).to(BF16)
    binding.spec_cache_write(cache, table, ints(0), new.cuda(), new.cuda())
    back = binding.spec_cache_read(cache, table, None, None, 300)[0]
    near = (back.cpu().double() - new.double()).abs() <= 2.0 ** -4 * new.double().abs() + 2.0 ** -10 * 0.02
    assert near.all()
    kept = [t.view(torch.uint8)[[7, pages - 3, pages - 1]].cpu().view(torch.float8_e4m3fn) for t in (k, v)]
    state = (*kept, cache.k_scale[[7, pages - 3, pages - 1]].cpu(),
             cache.v_scale[[7, pages - 3, pages - 1]].cpu(), torch.tensor([[2, 1, 0]], dtype=torch.int32))
    for N in (1, 40):
        q = torch.randn((1, N, 4, D), generator=g).to(BF16)
        got = binding.spec_cache_attention(q.cuda(), cache, table, ints(300 - N))[0].cpu().double()
        o, _, tol, _ = ref.attention(ref.Cache(*state, "e4m3"), 0, 300 - N, N, q[0].double(), None, D ** -0.5)
        assert torch.all((got[0] - o).abs() <= tol + 2.0 ** -8 * o.abs())
    assert binding.spec_get_status() == 0


# ----------------------------------------------------------------- commit
def paths(parent, tokens, node):
    at, ids = node, []
    while at >= 0:
        ids.insert(0, at)
        at = int(parent[at])
    return ids, [int(tokens[i]) for i in ids[1:]]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("page,D", [(16, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("N,shared", [(1, False), (8, True), (63, False), (200, True)])
def test_commit(kind, page, D, N, shared):
    B, Hk = 5, 2
    g = torch.Generator().manual_seed(N + page)
    parent = random_trees(g, 1 if shared else B, N).expand(B, N).contiguous()
    tokens = torch.randint(0, 6, (B, N), generator=g, dtype=torch.int32)   # equal tokens among siblings
    ctx = [0, 1, page - 1, page, 2 * page + 5]
    state = make_cache(B, 2 * page + 5 + N, Hk, page, D, kind, N)
    P = max(len(paths(parent[b], tokens[b], i)[0]) for b in range(B) for i in range(N))
    path, length = torch.full((B, P), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    want = ref.Cache(*state, kind)
    want_index = torch.full((B, P), -1, dtype=torch.int32)
    for b in range(B):
        node = N - 1 if b == 0 else int(torch.randint(0, N, (1,), generator=g))
        toks = paths(parent[b], tokens[b], node)[1]
        length[b] = len(toks) + 1
        path[b, :len(toks)] = torch.tensor(toks, dtype=torch.int32)
        path[b, len(toks)] = 5                        # the bonus token
        ids = next(p for p, t in (paths(parent[b], tokens[b], i) for i in range(N)) if t == toks)
        want_index[b, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        first = next((i for i, n in enumerate(ids) if i != n), len(ids))
        for t in (0, 1):
            rows = [want.row(t, b, ctx[b] + n) for n in ids[first:]]
            if rows:
                want.put(t, b, ctx[b] + first, torch.stack(rows), False)
    cache, table = on_gpu(state)
    index, new = binding.spec_cache_commit(cache, table, ints(*ctx), parent[0].cuda() if shared else parent.cuda(), tokens.cuda(),
                                           path.cuda(), length.cuda())
    assert binding.spec_get_status() == 0
    assert torch.equal(index.cpu(), want_index)
    assert new.tolist() == [c + int(n) for c, n in zip(ctx, length)]
    same_state(cache, want)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("page,D", [(16, 128), (32, 64)])
def test_commit_of_any_scales_and_codes(kind, page, D):
    """Scales that are no powers of two, zero, minus zero and so large that products overflow; codes that the write
    never makes (NaN, -128): every step in 32 bits, bit for bit."""
    B, N, Hk, ctx = 4, 90, 2, [5, 0, 20, 31]
    g = torch.Generator().manual_seed(page)
    state = list(make_cache(B, 31 + N, Hk, page, D, kind, 3))
    odd = 0x7f if kind == "e4m3" else 0x80
    for t in (0, 1):
        raw = state[t].view(torch.uint8)
        raw[torch.rand(raw.shape, generator=g) < 0.01] = odd
        scale = state[2 + t]
        scale *= 1 + torch.rand(scale.shape, generator=g)
        pick = torch.rand(scale.shape, generator=g)
        scale[pick < 0.3] = 1.37 * 2.0 ** 122
        scale[pick < 0.15] = 0.0
        scale[pick < 0.07] = -0.0
    parent = torch.arange(-3, N - 3, dtype=torch.int32).clamp(min=0)       # three chains from the root
    parent[0] = -1
    tokens = torch.arange(100, 100 + N, dtype=torch.int32).repeat(B, 1)
    ids = [[0] + list(range(s, N, 3))[:n] for s, n in ((2, 29), (3, 17), (2, 5), (3, 29))]
    path, length = torch.full((B, 31), -1, dtype=torch.int32), torch.tensor([len(i) for i in ids], dtype=torch.int32)
    want = ref.Cache(*state, kind)
    for b in range(B):
        path[b, :len(ids[b]) - 1] = 100 + torch.tensor(ids[b][1:], dtype=torch.int32)
        for t in (0, 1):
            rows = [want.row_f32(t, b, ctx[b] + n) for n in ids[b][1:]]
            want.put_f32(t, b, ctx[b] + 1, torch.stack(rows))
    cache, table = on_gpu(state)
    index, _ = binding.spec_cache_commit(cache, table, ints(*ctx), parent.cuda(), tokens.cuda(), path.cuda(), length.cuda())
    assert binding.spec_get_status() == 0
    for b in range(B):
        assert index[b, :len(ids[b])].tolist() == ids[b]
    same_state(cache, want)


def test_commit_leaves_failed_sequences_alone():
    N, D = 4, 64
    parent = ints(-1, 0, 0, 1).repeat(4, 1)
    parent[3, 2] = 3                                       # not a tree
    tokens = ints(0, 7, 8, 9).repeat(4, 1)
    path = torch.tensor([[8, 1, 0], [-1, -1, -1], [9, 1, 0], [8, 1, 0]], dtype=torch.int32, device="cuda")
    length = ints(2, -1, 2, 2)                             # sequence 2's path is not in its tree
    state = make_cache(4, 40, 1, 16, D, "e4m3", 2)
    cache, table = on_gpu(state)
    want = ref.Cache(*state, "e4m3")
    for t in (0, 1):
        want.put(t, 0, 10 + 1, want.row(t, 0, 10 + 2)[None], False)
    index, new = binding.spec_cache_commit(cache, table, ints(10, 11, 12, 13), parent, tokens, path, length)
    assert binding.spec_get_status() == 7                  # SPEC_ERR_PARENT, once
    assert index.tolist() == [[0, 2, -1]] + [[-1] * 3] * 3
    assert new.tolist() == [12, 11, 12, 13]
    same_state(cache, want)


# ------------------------------------------------------------- put together
def layer_step(cache, table, ctx, q, k, v, depth, mask, inv, counts=None):
    q, k = binding.spec_qk_norm_rope(q, k, inv, base=ctx, offset=depth)
    binding.spec_cache_write(cache, table, ctx, k, v, counts=counts)
    return binding.spec_cache_attention(q, cache, table, ctx, mask=mask, counts=counts)[0]


def test_an_accepted_path_continues_as_if_it_had_been_a_chain():
    """Verifying a tree and committing a path leaves the cache that verifying the path alone leaves (all values have
    one size, so that the blocks' scales agree)."""
    B, N, Hq, Hk, D, page = 3, 13, 8, 2, 128, 16
    g = torch.Generator().manual_seed(12)
    inv = 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)
    parent = ints(-1, 0, 0, 0, 1, 1, 2, 3, 4, 4, 6, 8, 9).repeat(B, 1)
    tokens = torch.arange(100, 100 + N, dtype=torch.int32, device="cuda").repeat(B, 1)
    mask, depth = binding.spec_tree_mask(parent)
    ctx = ints(30, 5, 16)
    x = {n: (torch.randint(0, 2, (B, N, h, D), generator=g) * 2 - 1).to(BF16).cuda() for n, h in (("q", Hq), ("k", Hk), ("v", Hk))}
    path = torch.tensor([[101, 104, 108, 111, 1], [102, 106, 2, -1, -1], [3, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    length = ints(5, 3, 1)
    ids = [[0, 1, 4, 8, 11], [0, 2, 6], [0]]
    state = make_cache(B, 60, Hk, page, D, "e4m3", 4, spread=0)
    cache, table = on_gpu(state)
    tree_out = layer_step(cache, table, ctx, x["q"], x["k"], x["v"], depth, mask, inv)
    index, new = binding.spec_cache_commit(cache, table, ctx, parent, tokens, path, length)
    for b in range(B):
        assert index[b, :len(ids[b])].tolist() == ids[b] and int(new[b]) == int(ctx[b]) + len(ids[b])
        chain_cache, chain_table = on_gpu([t[b:b + 1] if i == 4 else t for i, t in enumerate(state)])
        part = {n: t[b:b + 1, ids[b]].contiguous() for n, t in x.items()}
        out = layer_step(chain_cache, chain_table, ctx[b:b + 1], part["q"], part["k"], part["v"], None, None, inv)
        end = int(new[b])
        got = binding.spec_cache_read(cache, table[b:b + 1].contiguous(), None, None, end, dtype=F32)
        want = binding.spec_cache_read(chain_cache, chain_table, None, None, end, dtype=F32)
        for a, c in zip(got, want):
            # equal but for scales that other nodes raised: half a step of e4m3 each, or of its subnormals
            assert torch.all((a - c).abs() <= 2 * 2.0 ** -4 * c.abs() + 2.0 ** -8)
        # the same tokens seen by the same queries: fp16 weights and the output's rounding
        assert torch.all((tree_out[b, ids[b]].float() - out[0].float()).abs() <= 0.05)
    assert binding.spec_get_status() == 0


def test_a_layers_step_in_a_graph():
    B, N, Hq, Hk, D, page = 4, 6, 8, 2, 128, 32
    g = torch.Generator().manual_seed(2)
    inv = 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)
    state = make_cache(B, 500, Hk, page, D, "e4m3", 4)
    cache, table = on_gpu(state)
    ctx = ints(400, 3, 77, 0)
    q, k, v = (torch.randn((B, N, h, D), generator=g).to(BF16).cuda() for h in (Hq, Hk, Hk))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer_step(cache, table, ctx, q, k, v, None, None, inv)          # sizes the stream's workspace
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = layer_step(cache, table, ctx, q, k, v, None, None, inv)
    for seed in (5, 6):
        g = torch.Generator().manual_seed(seed)
        state = make_cache(B, 500, Hk, page, D, "e4m3", 4)
        fresh, _ = on_gpu(state)
        for n in ("k", "v", "k_scale", "v_scale"):
            getattr(cache, n).view(torch.uint8).copy_(getattr(fresh, n).view(torch.uint8))
        for t, h in ((q, Hq), (k, Hk), (v, Hk)):
            t.copy_(torch.randn((B, N, h, D), generator=g).to(BF16))
        ctx.copy_(ints(seed * 10, 450, 0, 31))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = layer_step(fresh, table, ctx, q, k, v, None, None, inv)
        assert torch.equal(out, want)
        assert torch.equal(cache.k.view(torch.uint8), fresh.k.view(torch.uint8))
    assert binding.spec_get_status(s) == 0 and binding.spec_get_status() == 0


def test_launch_failures_leave_the_next_call_right():
    state = make_cache(2, 3000, 1, 64, 128, "e4m3", 5)
    cache, table = on_gpu(state)
    q = torch.randn((2, 1, 4, 128), generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    ctx = ints(2900, 40)
    want = binding.spec_cache_attention(q, cache, table, ctx)[0]
    try:
        binding.spec_debug_fail_launch(1)
        with pytest.raises(binding.SpecError):
            binding.spec_cache_attention(q, cache, table, ctx)
    finally:
        binding.spec_debug_fail_launch(0)
    assert torch.equal(binding.spec_cache_attention(q, cache, table, ctx)[0], want)


def test_empty_calls():
    cache = SpecCache.empty(4, 2, 16, 64)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    zero = torch.empty((0,), dtype=torch.int32, device="cuda")
    q = torch.empty((0, 3, 4, 64), dtype=BF16, device="cuda")
    assert binding.spec_cache_attention(q, cache, none, zero)[0].shape == q.shape
    k = torch.empty((0, 3, 2, 64), dtype=BF16, device="cuda")
    binding.spec_cache_write(cache, none, zero, k, k)
    assert binding.spec_cache_read(cache, none, zero, None, 3)[0].shape == k.shape
    one = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    q = torch.empty((1, 0, 4, 64), dtype=BF16, device="cuda")
    assert binding.spec_cache_attention(q, cache, one, ints(0))[0].shape == q.shape
    assert binding.spec_qk_norm_rope(q, None)[0].shape == q.shape
    assert binding.spec_get_status() == 0


@pytest.mark.parametrize("kind,D", [("e4m3", 128), ("int8", 128), ("e4m3", 64), ("int8", 64)])
@pytest.mark.parametrize("N,G", [(2, 4), (3, 3), (2, 8), (17, 1), (23, 1), (3, 8), (6, 4), (25, 1), (4, 8), (43, 3), (16, 8), (37, 7)])
def test_attention_by_rows_per_kv_head(kind, D, N, G):
    """Each size class of rows (8, 16, 24, and tiles of 128), at its borders, over lengths on both sides of a tile and
    with blocks without values."""
    ctx = [0, 127 - N, 128, 1000, 2300]
    ctx[1] = max(ctx[1], 0)
    state = make_cache(len(ctx), 2300 + N, 2, 64, D, kind, N + G)
    state[3][::6] = 0
    g = torch.Generator().manual_seed(N + G)
    q = torch.randn((len(ctx), N, 2 * G, D), generator=g).to(BF16)
    check_attention(state, kind, ctx, None, q, None)
    parent = random_trees(g, len(ctx), N)
    check_attention(state, kind, ctx, [N, N, 1, N - 1, N], q, binding.spec_tree_mask(parent.cuda())[0].cpu())


@pytest.mark.parametrize("N", [1, 8])
def test_attention_of_many_sequences(N):
    """More sequences than a CTA has threads, many of them empty."""
    B, page, D = 2000, 16, 64
    state = make_cache(B, 48 + N, 1, page, D, "e4m3", 3)
    g = torch.Generator().manual_seed(5)
    ctx = torch.randint(0, 49, (B,), generator=g).tolist()
    counts = [N if i % 3 else 0 for i in range(B)]
    q = torch.randn((B, N, 4, D), generator=g).to(BF16)
    cache, table = on_gpu(state)
    out, lse = binding.spec_cache_attention(q.cuda(), cache, table, ints(*ctx), counts=ints(*counts), want_lse=True)
    assert binding.spec_get_status() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = torch.tensor(counts) == 0
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == -math.inf)
    want = ref.Cache(*state, "e4m3")
    for b in range(1, B, 31):
        o, l, to, tl = ref.attention(want, b, ctx[b], counts[b], q[b].double(), None, D ** -0.5)
        if counts[b]:
            assert torch.all((out[b] - o).abs() <= to + 2.0 ** -8 * o.abs()) and torch.all((lse[b] - l).abs() <= tl)


def test_two_streams_share_a_cache():
    """Calls on two streams at once read one cache, each with its own workspace."""
    state = make_cache(4, 5000, 2, 64, 128, "e4m3", 5)
    cache, table = on_gpu(state)
    g = torch.Generator().manual_seed(3)
    qs = [torch.randn((4, n, 8, 128), generator=g).to(BF16).cuda() for n in (1, 20)]
    ctx = ints(4900, 3000, 17, 0)
    want = [binding.spec_cache_attention(q, cache, table, ctx)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(binding.spec_cache_attention(q, cache, table, ctx, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))
    assert all(binding.spec_get_status(s) == 0 for s in streams)
