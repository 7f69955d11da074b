"""Attention of many short segments on the tile kernel: a CTA's stretch holds segments of one tile, in which one of its
two groups has no work, next to longer ones."""
import pytest
import torch

import cache_reference as ref
from sampling_row_online_gb300 import binding
from test_gpu_cache import BF16, ints, make_cache, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("lengths", [[3], [3, 119, 120, 3, 300], [100, 100, 100, 400], [119, 247, 0]])
def test_segments_of_one_tile_and_more(kind, D, lengths):
    B, N, Hq, Hk = 700, 9, 8, 2
    g = torch.Generator().manual_seed(len(lengths))
    ctx = [lengths[b % len(lengths)] for b in range(B)]
    state = make_cache(B, max(lengths) + N, Hk, 32, D, kind, 7)
    q = torch.randn((B, N, Hq, D), generator=g).to(BF16)
    cache, table = on_gpu(state)
    qc, cc = q.cuda(), ints(*ctx)
    out, lse = binding.spec_cache_attention(qc, cache, table, cc, want_lse=True)
    assert binding.spec_get_status() == 0
    for _ in range(5):
        again = binding.spec_cache_attention(qc, cache, table, cc, want_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert binding.spec_get_status() == 0
    out, lse, want = out.cpu().double(), lse.cpu().double(), ref.Cache(*state, kind)
    for b in range(0, B, 23):
        o, l, to, tl = ref.attention(want, b, ctx[b], N, q[b].double(), None, D ** -0.5)
        assert torch.all((out[b] - o).abs() <= to + 2.0 ** -8 * o.abs())
        assert torch.all((lse[b] - l).abs() <= tl)
