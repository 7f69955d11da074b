"""A page id outside the pool makes exactly the tokens NaN that see a slot of that page, whichever kernel attends."""
import math

import pytest
import torch

import cache_reference as ref
from sampling_row_online_gb300 import binding
from test_gpu_cache import BF16, F16, ints, make_cache, mask_of, on_gpu, random_trees

pytestmark = pytest.mark.gpu


def check(kind, D, dtype, N, Hq, Hk, ctx, counts, words, bad, page=16):
    """bad: {(sequence, block): page id}.  Page 0, which no sequence holds, is full of NaN codes."""
    B = len(ctx)
    state = list(make_cache(B, max(ctx) + N, Hk, page, D, kind, N + Hq))
    table = state[4]
    spare = sorted(set(range(len(state[0]))) - set(table.flatten().tolist()))[0]
    for t in (0, 1):                                      # whatever page 0 held goes to a page that nobody has
        state[t].view(torch.uint8)[spare] = state[t].view(torch.uint8)[0].clone()
        state[t].view(torch.uint8)[0] = 0x7f if kind == "e4m3" else 0x80
        state[2 + t][spare] = state[2 + t][0].clone()
    table[table == 0] = spare
    want = ref.Cache(*state, kind)
    broken = table.clone()
    for (b, block), page_id in bad.items():
        broken[b, block] = page_id
    q = torch.randn((B, N, Hq, D), generator=torch.Generator().manual_seed(N)).to(dtype)
    cache, _ = on_gpu(state)
    out, lse = binding.spec_cache_attention(q.cuda(), cache, broken.cuda(), ints(*ctx), counts=ints(*counts),
                                            mask=None if words is None else words.cuda(), want_lse=True)
    assert binding.spec_get_status() == 9                 # SPEC_ERR_PAGE
    assert binding.spec_get_status() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    some, other = 0, 0
    for b in range(B):
        m = None if words is None else mask_of(words[b], N)
        o, l, to, tl = ref.attention(want, b, ctx[b], counts[b], q[b].double(), m, D ** -0.5)
        for i in range(N):
            sees = set(range(ctx[b])) | {ctx[b] + j for j in range(counts[b]) if (j <= i if m is None else bool(m[i, j]))}
            if i >= counts[b]:
                sees = set()
            hit = any(s // page == block for (bb, block) in bad if bb == b for s in sees)
            if hit:
                some += 1
                assert torch.isnan(out[b, i]).all() and torch.isnan(lse[b, i]).all(), (b, i)
            else:
                other += 1
                tol = to[i] + ref.HALF_STEP[dtype] * o[i].abs() + (2.0 ** -25 if dtype == F16 else 1e-30)
                assert torch.all((out[b, i] - o[i]).abs() <= tol), (b, i)
                empty = torch.isinf(l[i])
                assert torch.equal(torch.isneginf(lse[b, i]), empty)
                assert torch.all(((lse[b, i] - l[i]).abs() <= tl[i])[~empty])
    assert some and other


# rows per kv head: 6 and 24 (streaming kernel), 32, 120 and 300 (tiles of 128 rows)
@pytest.mark.parametrize("kind,D,dtype", [("e4m3", 128, BF16), ("int8", 64, F16), ("e4m3", 64, F16)])
@pytest.mark.parametrize("N,Hq,Hk", [(6, 2, 2), (24, 1, 1), (32, 2, 2), (30, 8, 2), (100, 6, 2)])
def test_a_chain_sees_a_bad_page_from_its_first_slot_on(kind, D, dtype, N, Hq, Hk):
    ctx = [11, 130, 27, 0]
    last = [(c + N - 1) // 16 for c in ctx]               # the page of the last new token, and one in the middle
    bad = {(0, last[0]): -1, (1, last[1]): 10 ** 6, (3, last[3] // 2): -2 ** 31}
    check(kind, D, dtype, N, Hq, Hk, ctx, [N, N, N, N], None, bad)


@pytest.mark.parametrize("kind,D,dtype", [("e4m3", 128, BF16), ("int8", 64, F16)])
@pytest.mark.parametrize("N,Hq,Hk", [(20, 1, 1), (24, 2, 2), (40, 4, 2), (130, 4, 2)])
def test_a_tree_sees_a_bad_page_where_its_mask_does(kind, D, dtype, N, Hq, Hk):
    g = torch.Generator().manual_seed(N)
    words = binding.spec_tree_mask(random_trees(g, 3, N).cuda())[0].cpu()
    words[1, N // 2] = 0                                  # a node that sees its context only
    ctx, counts = [9, 0, 131], [N, N, N - 1]
    bad = {(0, (9 + N - 1) // 16): -1, (1, (N - 1) // 16): 10 ** 6, (2, (131 + N // 2) // 16): 2 ** 31 - 1}
    check(kind, D, dtype, N, Hq, Hk, ctx, counts, words, bad)


@pytest.mark.parametrize("N", [1, 30])
def test_a_bad_page_of_the_context_reaches_every_token(N):
    B, Hk, page, D = 2, 2, 32, 128
    state = make_cache(B, 200 + N, Hk, page, D, "e4m3", 5)
    state[4][1, 3] = -1
    cache, table = on_gpu(state)
    q = torch.randn((B, N, 4, D), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out, lse = binding.spec_cache_attention(q, cache, table, ints(200, 200), want_lse=True)
    assert binding.spec_get_status() == 9
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(out[1].float()).all() and torch.isnan(lse[1]).all()
    assert not math.isnan(float(out[0].float().sum()))
