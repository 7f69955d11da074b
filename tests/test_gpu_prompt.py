"""GPU parity of the attention over whole prompts against a plain 64-bit restatement, within counted roundings."""
import math

import pytest
import torch

import prompt_reference as ref
from sampling_row_online_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def tensors(T, Hq, Hk, D, dtype, seed, size=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    both = torch.randn((T, Hq + 2 * Hk, D), generator=g, device="cuda")
    both[:, :Hq] *= size
    both = both.to(dtype)
    return both[:, :Hq], both[:, Hq:Hq + Hk], both[:, Hq + Hk:]


def starts_of(lengths, first=0):
    s = [first]
    for n in lengths:
        s.append(s[-1] + n)
    return s


def check(q, k, v, starts, scale=None, **kw):
    on = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out, lse = binding.spec_prompt_attention(q, k, v, on, scale=scale, want_lse=True, **kw)
    assert binding.spec_get_status() == 0
    want, wlse, tol, tol_lse = ref.prompt_attention(q, k, v, starts, q.shape[-1] ** -0.5 if scale is None else scale)
    assert out.shape == q.shape and out.dtype == q.dtype and lse.shape == q.shape[:2]
    inside = torch.zeros(len(q), dtype=torch.bool, device="cuda")
    inside[starts[0]:starts[-1]] = True
    assert not out[~inside].any() and (lse[~inside] == -math.inf).all()
    off = (out.double() - want).abs()[inside]
    assert (off <= tol[inside]).all(), (off - tol[inside]).max().item()
    off = (lse.double() - wlse).abs()[inside]
    assert (off <= tol_lse[inside]).all(), off.max().item()
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (8, 2), (10, 2), (7, 1), (16, 2), (40, 1)])
def test_group_sizes(dtype, D, Hq, Hk):
    lengths = [1, 0, 33, 129, 300]
    q, k, v = tensors(sum(lengths), Hq, Hk, D, dtype, Hq + D)
    check(q, k, v, starts_of(lengths))


@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [63, 64, 65], [127, 128, 129], [255, 256, 257], [0, 0, 5, 0], [511, 1, 513],
                                     [1023, 1, 1, 1], [2051]], ids=str)
@pytest.mark.parametrize("Hq,Hk,D", [(4, 4, 128), (8, 2, 128), (4, 2, 64)])
def test_lengths(lengths, Hq, Hk, D):
    q, k, v = tensors(sum(lengths), Hq, Hk, D, BF16, sum(lengths))
    check(q, k, v, starts_of(lengths))


def test_many_heads_for_one():
    """More query heads than a tile has rows share a kv head."""
    q, k, v = tensors(70, 260, 2, 64, BF16, 1)
    check(q, k, v, starts_of([50, 20]))
    q, k, v = tensors(40, 131, 1, 128, F16, 2)             # a prime number of them
    check(q, k, v, starts_of([7, 33]))


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 9, (1500,), generator=g).tolist()
    q, k, v = tensors(sum(lengths), 4, 2, 64, BF16, 3)
    check(q, k, v, starts_of(lengths))


def test_one_sequence_over_many_ctas():
    q, k, v = tensors(5003, 2, 1, 128, BF16, 4)
    check(q, k, v, [0, 5003])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scores_that_rise_and_fall(dtype):
    """The running maximum moves far up, late, and by steps; weights of early tokens vanish beside later ones."""
    T, Hq, Hk, D = 900, 4, 2, 64
    q, k, v = tensors(T, Hq, Hk, D, dtype, 5)
    q, k = torch.zeros_like(q.contiguous()), torch.zeros_like(k.contiguous())
    q[..., 0] = 1
    ramp = torch.linspace(-60, 60, T, device="cuda")
    k[:, 0, 0] = ramp.to(dtype)
    k[:, 1, 0] = ramp.flip(0).to(dtype)
    check(q, k, v, [0, 600, 900], scale=1.0)
    check(q, k, v, [0, 600, 900], scale=-1.0)
    k[:, 0, 0] = 0
    k[513, 0, 0] = 80
    check(q, k, v, [0, 900], scale=1.0)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25])
def test_scales(scale):
    q, k, v = tensors(300, 4, 2, 128, BF16, 6, size=0.3)
    check(q, k, v, [0, 100, 300], scale=scale)


@pytest.mark.parametrize("layout", ["one_projection", "heads_first", "odd_offset", "shared_keys", "every_other_row", "slice_of_heads"])
@pytest.mark.parametrize("D", [64, 128])
def test_any_strides(layout, D):
    T, Hq, Hk = 261, 6, 3
    q, k, v = tensors(T, Hq, Hk, D, BF16, 7)
    if layout == "heads_first":
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    elif layout == "odd_offset":
        q, k, v = (torch.cat([x, x[..., :1]], -1)[..., 1:] for x in (q, k, v))
    elif layout == "shared_keys":
        k, v = (x[:, :1].expand(T, Hk, D) for x in (k, v))
    elif layout == "every_other_row":
        q, k, v = (x.repeat_interleave(2, 0)[::2] for x in (q, k, v))
    elif layout == "slice_of_heads":
        q, k, v = q[:, 1:4], k[:, 2:], v[:, 2:]
    check(q, k, v, [3, 100, 250])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_what_a_row_does_not_see_does_not_matter(dtype, junk):
    """Rows of no sequence, later rows of the same sequence, and other sequences may hold anything."""
    starts = [5, 70, 333, 400]
    T, Hq, Hk, D = 420, 8, 2, 128
    q, k, v = tensors(T, Hq, Hk, D, dtype, 8)
    clean = check(q, k, v, starts)
    for x in (q, k, v):
        x[:5] = junk
        x[400:] = junk
    again = binding.spec_prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), want_lse=True)
    assert torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])
    # a token in the middle of a sequence: those before it, and the other sequences, stay as they are
    for t in (200, 332, 70):
        kk, vv = k.clone(), v.clone()
        vv[t, 0, 3] = junk
        kk[t, 1, 5] = junk
        on = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out, lse = binding.spec_prompt_attention(q, kk, vv, on, want_lse=True)
        assert binding.spec_get_status() == 0
        other = torch.ones(T, dtype=torch.bool, device="cuda")
        other[t:333] = False
        assert torch.equal(out[other], clean[0][other]) and torch.equal(lse[other], clean[1][other])
        # a value that is not finite reaches its own column of the rows that see it, and no other
        seen = out[t:333, :4]
        columns = torch.ones(D, dtype=torch.bool, device="cuda")
        columns[3] = False
        assert not seen[..., 3].isfinite().any()
        if junk == junk:
            assert (seen[..., 3] == junk).all()
        assert torch.equal(seen[..., columns], clean[0][t:333, :4][..., columns])
        assert torch.equal(lse[t:333, :4], clean[1][t:333, :4])
        if junk != junk:
            assert out[t:333, 4:].isnan().all()


def test_starts_that_do_not_ascend():
    q, k, v = tensors(50, 4, 2, 64, BF16, 9)
    for bad in ([0, 30, 20, 50], [-1, 50], [0, 51], [10, 5], [0, 2 ** 31 - 1, 50]):
        out, lse = binding.spec_prompt_attention(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), want_lse=True)
        assert binding.spec_get_status() == 1
        assert out.isnan().all() and lse.isnan().all()
    check(q, k, v, [0, 50])


def test_no_sequences():
    q, k, v = tensors(50, 4, 2, 64, BF16, 9)
    for starts in ([0], [7], [0, 0], [50, 50, 50]):
        check(q, k, v, starts)
    check(q[:0], k[:0], v[:0], [0, 0])


def test_repeats_itself_and_takes_an_output():
    q, k, v = tensors(3001, 8, 2, 128, BF16, 10)
    starts = torch.tensor([0, 1234, 3001], dtype=torch.int32, device="cuda")
    out, lse = binding.spec_prompt_attention(q, k, v, starts, want_lse=True)
    mine = torch.full_like(out, 7.0)
    for _ in range(3):
        again, l2 = binding.spec_prompt_attention(q, k, v, starts, want_lse=True, out=mine)
        assert again is mine and torch.equal(out, again) and torch.equal(lse, l2)
    only, none = binding.spec_prompt_attention(q, k, v, starts)
    assert none is None and torch.equal(only, out)
    assert binding.spec_get_status() == 0


def test_captured_and_on_another_stream():
    """A captured call follows new inputs and new starts; two streams do not share what they work on."""
    T = 2000
    q, k, v = (x.contiguous() for x in tensors(T, 8, 2, 128, BF16, 11))
    starts = torch.tensor([0, 700, 2000], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.spec_prompt_attention(q, k, v, starts, want_lse=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = binding.spec_prompt_attention(q, k, v, starts, want_lse=True)
    for seed, s in ((12, [0, 1, 2000]), (13, [10, 1000, 1990])):
        q2, k2, v2 = tensors(T, 8, 2, 128, BF16, seed)
        q.copy_(q2), k.copy_(k2), v.copy_(v2)
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        more = [binding.spec_prompt_attention(q, k, v, starts, want_lse=True) for _ in range(4)]  # beside the replay
        torch.cuda.synchronize()
        for o, l2 in more:
            assert torch.equal(o, out) and torch.equal(l2, lse)
        check(q, k, v, s)
    assert binding.spec_get_status(side) == 0
