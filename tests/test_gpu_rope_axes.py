"""GPU parity of the rotation with several axes: against a plain 64-bit restatement, and bit for bit against the rotation
with one axis where all axes stand at the same position."""
import pytest
import torch

import prompt_reference as ref
from cache_reference import HALF_STEP
from sampling_row_online_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def inputs(B, N, Hq, Hk, D, dtype, rot, axes, seed, far=100000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn((B, N, h, D), generator=g, device="cuda").mul_(3).to(dtype) for h in (Hq, Hk))
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    positions = torch.randint(-5, far, (B, N, axes), generator=g, device="cuda", dtype=torch.int32)
    base = torch.randint(0, far, (B,), generator=g, device="cuda", dtype=torch.int32)
    inv_freq = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))
    axis = torch.randint(0, axes, (rot // 2,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return q, k, w, positions, base, inv_freq, axis


def close(got, x, weight, positions, axis, inv_freq, rot, pairs, norm):
    want = ref.rotate(x, weight, positions, axis, inv_freq, rot, pairs, norm, 1e-6)
    # both elements of a pair: norm, weight, products with sine and cosine, each a few roundings of 32 bits, an angle to
    # 2^-24 of a half turn; then one rounding to the type
    size = want.abs().clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        size[..., a] = size[..., b] = torch.hypot(want[..., a], want[..., b])
    off = (got.double() - want).abs()
    tol = 2.0 ** -19 * size + HALF_STEP[got.dtype] * (want.abs() + 2.0 ** -19 * size) + 2.0 ** -25 * (got.dtype == F16) + 1e-38
    assert (off <= tol).all(), (off - tol).max().item()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (256, 256), (80, 40), (96, 30), (6, 2)])
@pytest.mark.parametrize("axes", [1, 3, 8])
def test_axes(dtype, pairs, D, rot, axes):
    B, N, Hq, Hk = 3, 17, 4, 2
    q, k, w, positions, base, inv_freq, axis = inputs(B, N, Hq, Hk, D, dtype, rot, axes, D + rot + axes)
    oq, ok = binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis, positions, base=base, q_weight=w[0], k_weight=w[1], pairs=pairs)
    where = positions.long() + base.long()[:, None, None]
    close(oq, q, w[0], where, axis, inv_freq, rot, pairs, True)
    close(ok, k, w[1], where, axis, inv_freq, rot, pairs, True)
    oq, ok = binding.spec_qk_norm_rope_axes(q, None, inv_freq, axis, positions, norm=False, pairs=pairs)
    assert ok is None
    close(oq, q, None, positions.long(), axis, inv_freq, rot, pairs, False)
    assert binding.spec_get_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("B,N,D,rot", [(1, 1, 128, 128), (5, 400, 128, 128), (2, 33, 80, 60)])
def test_one_position_on_every_axis_is_the_plain_rotation(dtype, pairs, B, N, D, rot):
    q, k, w, positions, base, inv_freq, axis = inputs(B, N, 8, 2, D, dtype, rot, 3, N)
    offset = positions[..., 0].contiguous()
    same = offset[..., None].expand(B, N, 3).contiguous()
    want = binding.spec_qk_norm_rope(q, k, inv_freq, base=base, offset=offset, q_weight=w[0], k_weight=w[1], pairs=pairs)
    got = binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis, same, base=base, q_weight=w[0], k_weight=w[1], pairs=pairs)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_far_positions_strides_and_in_place():
    B, N, Hq, Hk, D = 2, 9, 4, 2, 64
    q, k, w, positions, _, inv_freq, axis = inputs(B, N, Hq, Hk, D, BF16, D, 4, 1, far=2 ** 31 - 1)
    both = torch.cat([q, k], 2)
    q, k = both[:, :, :Hq], both[:, :, Hq:]
    before = both.clone()
    out = binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis, positions, q_weight=w[0], k_weight=w[1], out_q=q, out_k=k)
    assert out[0] is q and out[1] is k
    close(q, before[:, :, :Hq], w[0], positions.long(), axis, inv_freq, D, False, True)
    close(k, before[:, :, Hq:], w[1], positions.long(), axis, inv_freq, D, False, True)


def test_no_rotation_and_wrong_tensors():
    q, k, w, positions, base, inv_freq, axis = inputs(1, 5, 2, 1, 64, BF16, 64, 3, 2)
    none = torch.zeros(0, dtype=torch.int32)
    a = binding.spec_qk_norm_rope_axes(q, k, torch.zeros(0, dtype=torch.float64), none, positions, q_weight=w[0], k_weight=w[1])
    b = binding.spec_qk_norm_rope(q, k, None, q_weight=w[0], k_weight=w[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis[:-1], positions)
    with pytest.raises(ValueError):
        binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis.cuda(), positions)
    with pytest.raises(ValueError):
        binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis, positions[:, :4])
    with pytest.raises(TypeError):
        binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis, positions.long())
    with pytest.raises(binding.SpecError):
        binding.spec_qk_norm_rope_axes(q, k, inv_freq, axis + 3, positions)
