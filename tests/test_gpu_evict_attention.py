"""Attention over what an eviction has left: against a plain 64-bit softmax over the rows that were kept, and against the
attention before it where the slots that went had no weight."""
import pytest
import torch

from cache_reference import HALF_STEP
from sampling_row_online_gb300 import SpecCache, binding

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def inputs(B, ctx, Hk, G, D, seed):
    """Keys of which a quarter count and the others score 150 below them; in every row one element of the largest size, which
    no query sees (keys) or which all rows share (values), so that every block has the same scale wherever its rows come
    from."""
    g = torch.Generator().manual_seed(seed)
    busy = torch.rand((B, ctx, Hk), generator=g) < 0.25
    keys, values = torch.randn((B, ctx + 1, Hk, D), generator=g) * 0.3, torch.randn((B, ctx + 1, Hk, D), generator=g).clamp(-3.9, 3.9)
    keys[..., 0] = 0
    keys[:, :ctx, :, 0] = -40.0 * ~busy
    keys[..., 1], values[..., 0] = 40.0, 4.0
    q = torch.randn((B, 1, Hk * G, D), generator=g)
    q[..., 0], q[..., 1] = 3.75 * D ** 0.5, 0.0
    return busy, keys.to(BF16).cuda(), values.to(BF16).cuda(), q.to(BF16).cuda()


def plain(q, k, v):
    """One sequence and one token in 64 bits: (out [Hq, D], what it may be off by); k and v [slots, Hk, D]."""
    Hq, D = q.shape
    G = Hq // k.shape[1]
    out, tol = torch.zeros((2, Hq, D), dtype=torch.float64, device=q.device)
    for h in range(Hq):
        qq, kk, vv = q[h].double(), k[:, h // G].double(), v[:, h // G].double()
        p = (kk @ qq * D ** -0.5).softmax(0)
        # a score: D products in 32 bits and a few roundings; weights once to fp16, the output once to bf16
        off = (D + 8) * 2.0 ** -24 * (kk.abs() @ qq.abs()).max() * D ** -0.5 + 2.0 ** -16
        out[h] = p @ vv
        spread = (2.0 ** -11 + 2 * off) * (p @ vv.abs())
        tol[h] = spread + HALF_STEP[BF16] * (out[h].abs() + spread) * 1.01
    return out, tol


def rows(cache, table, n):
    """[B, n, Hk, D] in 32 bits: the keys and the values of every sequence's first n slots."""
    return binding.spec_cache_read(cache, table, None, None, n, dtype=torch.float32)


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("D,page,G", [(64, 16, 4), (128, 32, 1), (128, 64, 7)])
def test_attention_over_what_is_left(kind, D, page, G):
    B, Hk, ctx = 2, 2, 200
    busy, keys, values, q = inputs(B, ctx, Hk, G, D, D + G)
    per = -(-(ctx + 1) // page)
    cache = SpecCache.empty(B * per, Hk, page, D, dtype=kind)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, per).cuda()
    lens = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    binding.spec_cache_write(cache, table, torch.zeros_like(lens), keys, values)
    out, lse = binding.spec_cache_attention(q, cache, table, lens, want_lse=True)
    k0, v0 = rows(cache, table, ctx + 1)
    weights = torch.zeros((B, Hk, per * page), device="cuda")
    binding.spec_cache_weights(q, cache, table, lens, lse, weights)
    keep = int(busy.sum(1).max()) + 9
    assert keep < ctx // 2
    index, left = binding.spec_cache_evict(cache, table, lens, weights, keep, last=8)
    assert left.tolist() == [keep] * B
    binding.spec_cache_write(cache, table, left, keys[:, ctx:], values[:, ctx:])
    again, _ = binding.spec_cache_attention(q, cache, table, left)
    k1, v1 = rows(cache, table, keep + 1)
    assert binding.spec_get_status() == 0
    for b in range(B):
        kept = torch.cat([index[b].long(), torch.full((Hk, 1), ctx, device="cuda")], 1)  # and the new token
        for h in range(Hk):
            assert set(busy[b, :, h].nonzero()[:, 0].tolist()) <= set(kept[h].tolist())
            # no block's scale differs, so the rows are the same bits
            assert torch.equal(k1[b, :, h], k0[b, kept[h], h]) and torch.equal(v1[b, :, h], v0[b, kept[h], h])
        k, v = (torch.stack([x[b, kept[h], h] for h in range(Hk)], 1) for x in (k0, v0))
        want, tol = plain(q[b, 0], k, v)
        off = (again[b, 0].double() - want).abs()
        assert (off <= tol).all(), (off - tol).max().item()
        # what went had no weight: e to the -100 at most
        full, more = plain(q[b, 0], k0[b], v0[b])
        assert ((out[b, 0].double() - full).abs() <= more).all()
        assert ((again[b, 0].double() - out[b, 0].double()).abs() <= tol + more + 1e-30).all()
        # the bounds tell other rows from these: nothing, and the values in another order
        assert (want.abs() > tol).any(-1).all()
        assert ((plain(q[b, 0], k, v.roll(1, 0))[0] - want).abs() > tol).any(-1).all()
