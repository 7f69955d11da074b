"""The attention over whole prompts where segments are shared between CTAs: heads per kv head that do not divide a tile, so
that row tiles begin and end inside token tiles, and batches of long and short sequences."""
import pytest
import torch

from sampling_row_online_gb300 import binding
from test_gpu_prompt import BF16, F16, check, starts_of, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2049, 2687, 3333, 4500])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(3, 1, 128, BF16), (5, 1, 64, BF16), (7, 1, 128, F16), (6, 2, 64, F16), (11, 1, 128, BF16),
                                           (13, 1, 64, F16), (48, 1, 128, BF16), (25, 5, 64, BF16)])
def test_groups_that_do_not_divide_a_tile(Hq, Hk, D, dtype, T):
    q, k, v = tensors(T, Hq, Hk, D, dtype, T + Hq)
    check(q, k, v, [0, T])


@pytest.mark.parametrize("Hq,Hk,D,dtype", [(4, 4, 128, BF16), (8, 2, 64, F16), (7, 1, 128, BF16), (10, 2, 64, BF16), (130, 1, 64, F16)])
def test_long_and_short_sequences(Hq, Hk, D, dtype):
    g = torch.Generator().manual_seed(Hq)
    lengths = torch.randint(1, 300, (20,), generator=g).tolist()
    lengths[7], lengths[11], lengths[12] = 3001, 0, 2048
    q, k, v = tensors(sum(lengths) + 9, Hq, Hk, D, dtype, Hq)
    starts = starts_of(lengths, first=4)
    out, lse = check(q, k, v, starts)
    # the same again, and each sequence by itself to within what is rounded
    on = torch.tensor(starts, dtype=torch.int32, device="cuda")
    again, lse2 = binding.spec_prompt_attention(q, k, v, on, want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    lo, hi = starts[7], starts[8]
    check(q[lo:hi], k[lo:hi], v[lo:hi], [0, hi - lo])


@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (4, 4, 64)])
def test_as_many_sequences_as_can_be(Hq, Hk, D):
    """65535 of them, nearly all empty."""
    lengths = [0] * 65535
    lengths[3], lengths[40000], lengths[40001], lengths[65534] = 5, 150, 1, 33
    q, k, v = tensors(sum(lengths) + 2, Hq, Hk, D, BF16, D)
    on = torch.tensor(starts_of(lengths, first=1), dtype=torch.int32, device="cuda")
    out, lse = binding.spec_prompt_attention(q, k, v, on, want_lse=True)
    few = check(q, k, v, [1, 6, 156, 157, 190])
    assert torch.equal(out, few[0]) and torch.equal(lse, few[1])
    assert binding.spec_get_status() == 0
