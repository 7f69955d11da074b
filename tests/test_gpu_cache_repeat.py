"""Each operator around the 8-bit cache, called again on the same inputs and state, gives the same bytes: no result depends
on the order in which CTAs run."""
import pytest
import torch

from sampling_row_online_gb300 import binding
from test_gpu_cache import BF16, ints, make_cache, on_gpu, random_trees

pytestmark = pytest.mark.gpu

B, Hk, D, page, N = 24, 4, 128, 32, 60


def twice(fn):
    a, b = ([t.clone() for t in fn()] for _ in range(2))
    assert binding.spec_get_status() == 0
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def fresh(kind):
    return on_gpu(make_cache(B, 2000 + N, Hk, page, D, kind, 3))


def state(cache):
    return cache.k, cache.v, cache.k_scale, cache.v_scale


def normal(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


CTX = [(83 * b) % 2000 for b in range(B)]


@pytest.mark.parametrize("pairs", [False, True])
def test_norms_and_rotation(pairs):
    q, k = normal(B, N, 16, D), normal(B, N, Hk, D, seed=2)
    inv = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    twice(lambda: binding.spec_qk_norm_rope(q, k, inv, base=ints(*CTX), pairs=pairs))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_write_and_read(kind):
    k, v = normal(B, N, Hk, D) * 20, normal(B, N, Hk, D, seed=2)

    def run():
        cache, table = fresh(kind)
        binding.spec_cache_write(cache, table, ints(*CTX), k, v)
        return state(cache) + binding.spec_cache_read(cache, table, None, ints(*(c + N for c in CTX)), 2000 + N)

    twice(run)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_commit(kind):
    parent = random_trees(torch.Generator().manual_seed(4), B, N)
    tokens = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    path, length = torch.full((B, N), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        at, ids = N - 1 - b, []
        while at > 0:
            ids.insert(0, at)
            at = int(parent[b, at])
        path[b, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        length[b] = len(ids) + 1

    def run():
        cache, table = fresh(kind)
        moved = binding.spec_cache_commit(cache, table, ints(*CTX), parent.cuda(), tokens.cuda(), path.cuda(), length.cuda())
        return state(cache) + moved

    twice(run)


@pytest.mark.parametrize("heads,nodes", [(16, 1), (16, 6), (32, 60)])
def test_attention(heads, nodes):
    cache, table = fresh("e4m3")
    q = normal(B, nodes, heads, D)
    twice(lambda: binding.spec_cache_attention(q, cache, table, ints(*CTX), want_lse=True))
