"""The limit on a call's work, which goes by the table's width and not by what is used of it."""
import math

import pytest
import torch

from sampling_row_online_gb300 import binding
from test_gpu_cache import BF16, ints, make_cache, on_gpu

pytestmark = pytest.mark.gpu


def test_a_table_far_wider_than_the_call():
    """What counts against the limit on a call's work is tiles of 128 rows and 128 tokens: 32768 tokens of 64 heads in a
    table of 2^21 slots, of which a few are used."""
    Hk, D, page, N, per = 64, 64, 128, 32768, 2 ** 14
    state = make_cache(1, 300, Hk, page, D, "int8", 3)
    cache, small = on_gpu(state)
    table = torch.full((1, per), -1, dtype=torch.int32, device="cuda")
    table[:, :small.shape[1]] = small
    row = torch.randn((1, 40, Hk, D), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    want = binding.spec_cache_attention(row, cache, small, ints(200), want_lse=True)
    q = torch.zeros((1, N, Hk, D), dtype=BF16, device="cuda")
    q[:, :40] = row
    out, lse = binding.spec_cache_attention(q, cache, table, ints(200), counts=ints(40), want_lse=True)
    assert binding.spec_get_status() == 0
    assert torch.equal(out[:, :40], want[0]) and torch.equal(lse[:, :40], want[1])
    assert torch.all(out[:, 40:] == 0) and torch.all(lse[:, 40:] == -math.inf)
    for per in (2 ** 17, 2 ** 20):                        # 2^31 tiles and more are refused
        with pytest.raises(binding.SpecError):
            binding.spec_cache_attention(q, cache, torch.zeros((1, per), dtype=torch.int32, device="cuda"), ints(0), counts=ints(40))
