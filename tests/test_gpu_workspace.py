"""A captured call keeps the workspace that it was captured with: replays are right after any other calls on the same
stream, of whatever size.  Each test starts from no workspace, so that the later calls do outgrow the captured one's."""
import pytest
import torch

from sampling_row_online_gb300 import SpecCache, binding
from sampling_row_online_gb300.workloads import NgramWorkload, Workload, make_chain, make_contexts

pytestmark = pytest.mark.gpu


@pytest.fixture
def stream():
    torch.cuda.synchronize()
    binding.spec_shutdown()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    yield s
    torch.cuda.synchronize()


def captured(fn, s):
    with torch.cuda.stream(s):
        fn()                                        # sizes the workspace
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fn()
    return g


def attention(N, Hq, B=3, L=3000, Hk=2, D=128, page=64):
    """A call's inputs over contexts long enough that many CTAs share a segment."""
    g = torch.Generator(device="cuda").manual_seed(N * Hq)
    per = -(-(L + N) // page)
    codes = [torch.randn((B * per, Hk, page, D), generator=g, device="cuda").mul(60).to(torch.float8_e4m3fn) for _ in range(2)]
    cache = SpecCache(*codes, *(torch.full((B * per, Hk), 2.0 ** -6, device="cuda") for _ in range(2)))
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    ctx = torch.tensor([L, L // 2, 5], dtype=torch.int32, device="cuda")
    q = torch.randn((B, N, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    return lambda s: binding.spec_cache_attention(q, cache, table, ctx, out=out, stream=s), out


def spoil():
    """Memory that the driver could have handed out again, with contents that a stale pointer would meet."""
    return [torch.full((n,), 0x7f7f7f7f, dtype=torch.int32, device="cuda") for n in (152, 304, 1 << 12, 1 << 20, 1 << 20, 5 << 20)]


@pytest.mark.parametrize("first,then", [((1, 8), (20, 32)),      # pieces grow from the streaming to the tile kernel
                                        ((20, 32), (1, 8)),      # counters grow from one to two CTAs per SM
                                        ((1, 8), (6, 8)), ((6, 8), (1, 8))])
def test_attention_replayed_after_other_sizes(stream, first, then):
    run, out = attention(*first)
    run(None)
    want = out.clone()
    torch.cuda.synchronize()
    g = captured(lambda: run(stream), stream)
    other, other_out = attention(*then)
    other(None)
    other_want = other_out.clone()
    torch.cuda.synchronize()
    for _ in range(3):
        other(stream)
        stream.synchronize()
        assert torch.equal(other_out, other_want)
        kept = spoil()
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            g.replay()
        stream.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 0x7f7f7f7f).all()) for t in kept)
    assert binding.spec_get_status(stream) == 0


def test_verification_replayed_after_larger_calls(stream):
    w = Workload("g", "chain", B=2, K=3, V=32000, dtype="bf16", T=0.8, data_seed=31)
    zt, zd, x = make_chain(w, device="cuda")
    out = torch.empty((w.B, w.K + 1), dtype=torch.int32, device="cuda")
    n = torch.empty((w.B,), dtype=torch.int32, device="cuda")
    want = binding.spec_verify(zt, zd, x, w.T, 9)
    torch.cuda.synchronize()
    g = captured(lambda: binding.spec_verify(zt, zd, x, w.T, 9, out_tokens=out, out_n_accepted=n, stream=stream), stream)
    big = Workload("g", "chain", B=32, K=5, V=128256, dtype="bf16", T=0.8, data_seed=32)
    bt, bd, bx = make_chain(big, device="cuda")
    attend, _ = attention(20, 32)
    torch.cuda.synchronize()
    for larger in (lambda: binding.spec_verify(bt, bd, bx, big.T, 9, stream=stream), lambda: attend(stream)):
        larger()
        stream.synchronize()
        kept = spoil()
        out.zero_(), n.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            g.replay()
        stream.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(n, want[1])
        assert all(bool((t == 0x7f7f7f7f).all()) for t in kept)
    assert binding.spec_get_status(stream) == 0


@pytest.mark.parametrize("L", [8192, 100000])        # a sequence's CTAs in a cluster, or joined by their counter
def test_drafting_replayed_after_larger_batches(stream, L):
    w = NgramWorkload("g", B=2, L=L, n_min=1, n_max=4, min_hits=1, K=5, V=32000, data_seed=41)
    tokens, lengths = make_contexts(w, device="cuda")
    draft = torch.empty((w.B, w.K), dtype=torch.int32, device="cuda")
    count = torch.empty((w.B,), dtype=torch.int32, device="cuda")
    want = binding.spec_ngram_propose(tokens, lengths, w.n_min, w.n_max, w.K)
    torch.cuda.synchronize()
    g = captured(lambda: binding.spec_ngram_propose(tokens, lengths, w.n_min, w.n_max, w.K, out_draft=draft, out_count=count,
                                                    stream=stream), stream)
    many = NgramWorkload("g", B=64, L=L, n_min=1, n_max=4, min_hits=1, K=5, V=32000, data_seed=42)
    t2, l2 = make_contexts(many, device="cuda")
    torch.cuda.synchronize()
    binding.spec_ngram_propose(t2, l2, w.n_min, w.n_max, w.K, stream=stream)
    stream.synchronize()
    kept = spoil()
    draft.zero_(), count.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        g.replay()
    stream.synchronize()
    assert torch.equal(draft, want[0]) and torch.equal(count, want[1])
    assert all(bool((t == 0x7f7f7f7f).all()) for t in kept)
    assert binding.spec_get_status(stream) == 0
