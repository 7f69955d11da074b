"""After every step of the example, the cache holds the rows of the committed tokens and of no others: keys and values of
one layer depend on a token and its position alone, so they are computed again in 64 bits from the tokens."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def rows_of(layer, tokens):
    """(keys, values) [T, kv_heads, dim] in 64 bits of tokens at positions 0, 1, ...  The layer rounds its products to bf16."""
    x = layer.embed[tokens].double()
    k, v = ((x @ w.double()).to(torch.bfloat16).double().view(len(tokens), layer.kv_heads, layer.dim) for w in (layer.wk, layer.wv))
    k = k / (k.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    f = torch.arange(len(tokens), device="cuda").double()[:, None] * layer.inv_freq.cuda()
    c, s = f.cos()[:, None], f.sin()[:, None]
    a, b = k[..., :layer.dim // 2], k[..., layer.dim // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1), v


def off(got, want, scale, kind):
    """Rows [T] of which some element is farther off than its roundings allow; scale [kv_heads, 1]: the largest of any block
    so far."""
    # keys and values leave a product as bf16, of which two may be a step apart: 2 2^-8 of the row's largest, which the keys'
    # rotation of pairs makes 2 sqrt(2) 2^-8, and its own rounding another 2^-8; the code's half step of a value so far off
    size = 5 * 2.0 ** -8 * want.abs().amax(-1, keepdim=True)
    # half a step of the code, at most once where the row was written and once where it was moved to, each time the block's scale
    # doubles: twice the last half step together (e4m3: of its least step; above it a power of two is exact)
    code = 2.0 ** -4 * want.abs() + 4 * 2.0 ** -10 * scale if kind == "e4m3" else 2 * scale
    return ((got - want).abs() > size + code).any(-1).any(-1)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("nodes,page", [(13, 32), (40, 16)])
def test_the_cache_holds_the_committed_tokens(monkeypatch, kind, nodes, page):
    import tree_step
    prompt, batch, seen, layers = 37, 3, [], []
    commit, build = tree_step.lib.spec_cache_commit, tree_step.Layer

    def spy(cache, table, ctx, parent, tokens, path, length):
        index, after = commit(cache, table, ctx, parent, tokens, path, length)
        rows = tree_step.lib.spec_cache_read(cache, table, None, after, int(after.max()), dtype=torch.float32)
        seen.append((after.tolist(), index.tolist(), rows, cache.k_scale[table.long()], cache.v_scale[table.long()]))
        return index, after

    def layer(*a, **kw):
        layers.append(build(*a, **kw))
        return layers[-1]

    first = []
    attend = build.logits
    monkeypatch.setattr(tree_step.lib, "spec_cache_commit", spy)
    monkeypatch.setattr(tree_step, "Layer", layer)
    monkeypatch.setattr(build, "logits", lambda self, cache, table, ctx, tokens, *a: first.append(tokens) or
                        attend(self, cache, table, ctx, tokens, *a))
    out = tree_step.decode(steps=10, batch=batch, nodes=nodes, prompt=prompt, kind=torch.int8 if kind == "int8" else torch.float8_e4m3fn, page=page)
    assert len(seen) == 10 and len(layers) == 1
    moved, largest = 0, [0, 0]
    for after, index, rows, *scales in seen:
        moved += sum(i > at for row in index for at, i in enumerate(row))
        largest = [torch.maximum(torch.as_tensor(m, device="cuda"), x.amax(1)).double() for m, x in zip(largest, scales)]
        for b in range(batch):
            n = after[b]
            tokens = torch.tensor(first[0][b].tolist() + out[b], device="cuda")[:n]
            for t, (got, want) in enumerate(zip(rows, rows_of(layers[0], tokens))):
                scale = largest[t][b][:, None]
                assert not off(got[b, :n].double(), want, scale, kind).any()
                # the bounds do tell rows apart: with the oracle one token further on
                assert off(got[b, :n].double(), want.roll(1, 0), scale, kind).float().mean() > 0.5
    assert moved > 0                                      # rows did have to move
