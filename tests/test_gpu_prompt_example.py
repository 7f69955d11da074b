"""The example runs the operators from a prompt to a cache within a budget together with the verification."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
def test_prompts_within_a_budget(kind):
    import prompt_step
    steps, keep, first, window = 5, 64, 4, 8
    done, kept, logits = prompt_step.serve(steps=steps, keep=keep, first=first, window=window, kind=kind)
    again, kept2, logits2 = prompt_step.serve(steps=steps, keep=keep, first=first, window=window, kind=kind)
    assert done == again and torch.equal(kept, kept2) and torch.equal(logits, logits2)       # deterministic
    assert all(len(row) >= steps + 1 for row in done)                                         # every pass commits a token
    lengths = [61, 99, 137]
    for b, n in enumerate(lengths):
        for h in range(kept.shape[1]):
            slots = [s for s in kept[b, h].tolist() if s >= 0]
            assert len(slots) == min(n, keep) and slots == sorted(set(slots)) and slots[-1] == n - 1
            if n > keep:
                assert slots[:first] == list(range(first)) and slots[-window:] == list(range(n - window, n))
    # a budget that holds everything changes nothing
    whole, _, _ = prompt_step.serve(steps=steps, keep=None, kind=kind)
    roomy, all_, _ = prompt_step.serve(steps=steps, keep=137, kind=kind)
    assert whole == roomy
    assert [int((all_[b, 0] >= 0).sum()) for b in range(3)] == lengths
    assert done[0] == whole[0]                                                                # the first prompt fits


def test_the_prompts_pass_is_the_layer_in_64_bits():
    """Rotation with three axes and causal attention, end to end, against plain 64-bit arithmetic on the same inputs."""
    import prompt_step
    import prompt_reference as ref
    import sampling_row_online_gb300 as lib
    layer = prompt_step.Layer(512, heads=8, kv_heads=2, dim=128)
    lengths, D = [50, 7, 77], 128
    T, starts = sum(lengths), [0, 50, 57, 134]
    tokens = torch.randint(0, 512, (T,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    positions = torch.cat([prompt_step.positions_of(n)[0] for n in lengths]).cuda()[None].contiguous()
    axis = (torch.arange(D // 2) % 3).to(torch.int32)
    x = layer.embed[tokens]
    q, k, v = ((x @ w).view(1, T, -1, D) for w in (layer.wq, layer.wk, layer.wv))
    rq, rk = lib.spec_qk_norm_rope_axes(q, k, layer.inv_freq, axis, positions, q_weight=layer.q_norm, k_weight=layer.k_norm)
    out, _ = lib.spec_prompt_attention(rq[0], rk[0], v[0], torch.tensor(starts, dtype=torch.int32, device="cuda"))
    assert lib.spec_get_status() == 0
    turned = [ref.rotate(t, w, positions.long(), axis, layer.inv_freq, D, False, True, 1e-6) for t, w in ((q, layer.q_norm), (k, layer.k_norm))]
    want = ref.prompt_attention(turned[0][0].to(torch.bfloat16), turned[1][0].to(torch.bfloat16), v[0], starts, D ** -0.5)
    # queries and keys are rounded to bf16 on both sides; where the two roundings differ, a score moves by a step of 2^-7
    # of one of its 128 products, and few do
    assert ((out.double() - want[0]).abs() <= 2 * want[2] + 2.0 ** -6 * v[0].double().abs().max()).all()
