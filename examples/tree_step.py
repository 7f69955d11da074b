"""Decoding with draft trees around an 8-bit paged key/value cache, with the library's calls only for what it does.

One attention layer with random weights stands in for the target model.  Each step drafts a tree of tokens for every
sequence, runs the layer over the tree's nodes (norms and rotation at the nodes' depths, the quantised write behind the
context, attention under the tree's mask), verifies the tree against the layer's logits, and commits the accepted path:
its rows move together in the cache and the context grows.

    python examples/tree_step.py [--steps 8] [--batch 4] [--nodes 13] [--int8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sampling_row_online_gb300 as lib  # noqa: E402


class Layer:
    """Queries, keys and values of a token's embedding, and logits of the attention's output."""

    def __init__(self, vocab, heads, kv_heads, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = heads * dim

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[0] ** -0.5).to(torch.bfloat16)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.embed = torch.randn((vocab, width), generator=g, device="cuda").to(torch.bfloat16)
        self.wq, self.wk, self.wv = weight(width, heads * dim), weight(width, kv_heads * dim), weight(width, kv_heads * dim)
        self.head = weight(width, vocab)
        self.q_norm, self.k_norm = (torch.ones(dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.inv_freq = 1e4 ** (-2 * torch.arange(dim // 2, dtype=torch.float64) / dim)

    def logits(self, cache, table, ctx, tokens, depth=None, mask=None):
        """[B, N, vocab] of tokens [B, N] behind the contexts; their keys and values are left in the cache."""
        B, N = tokens.shape
        x = self.embed[tokens.long()]
        q, k, v = ((x @ w).view(B, N, -1, self.dim) for w in (self.wq, self.wk, self.wv))
        q, k = lib.spec_qk_norm_rope(q, k, self.inv_freq, base=ctx, offset=depth, q_weight=self.q_norm, k_weight=self.k_norm)
        lib.spec_cache_write(cache, table, ctx, k, v)
        out, _ = lib.spec_cache_attention(q, cache, table, ctx, mask=mask)
        return (x + out.view(B, N, -1)) @ self.head


def draft_trees(layer, last, nodes, seed):
    """Trees [B, nodes] whose root is the last committed token: half of the nodes carry what the layer's head alone finds
    probable, the others any token."""
    B, vocab = last.shape[0], layer.embed.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    parent = torch.full((B, nodes), -1, dtype=torch.int32, device="cuda")
    tokens = torch.zeros((B, nodes), dtype=torch.int32, device="cuda")
    tokens[:, 0] = last
    for i in range(1, nodes):
        up = (i - 1) // 3                                  # three children each
        parent[:, i] = up
        guess = (layer.embed[tokens[:, up].long()] @ layer.head).topk(3).indices[:, (i - 1) % 3].to(torch.int32)
        other = torch.randint(0, vocab, (B,), generator=g, device="cuda", dtype=torch.int32)
        tokens[:, i] = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.5, guess, other)
    return parent, tokens


def decode(steps=8, batch=4, nodes=13, prompt=37, kind=torch.float8_e4m3fn, vocab=4096, page=32, seed=1):
    """Greedy decoding of `steps` tree steps.  Returns the committed tokens of each sequence (a list of lists)."""
    layer = Layer(vocab, heads=8, kv_heads=2, dim=128)
    g = torch.Generator(device="cuda").manual_seed(seed)
    most = prompt + (steps + 1) * nodes
    per = -(-most // page)
    cache = lib.SpecCache.empty(batch * per, layer.kv_heads, page, layer.dim, dtype=kind)
    tokens = torch.randint(0, vocab, (batch, prompt), generator=g, device="cuda", dtype=torch.int32)
    table = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32).view(batch, per)
    ctx = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    last = layer.logits(cache, table, ctx, tokens)[:, -1].argmax(-1).to(torch.int32)
    ctx = ctx + prompt
    out = [[int(t)] for t in last]
    for step in range(steps):
        parent, drafted = draft_trees(layer, last, nodes, seed * 1000 + step)
        mask, depth = lib.spec_tree_mask(parent)
        logits = layer.logits(cache, table, ctx, drafted, depth, mask)
        path, length = lib.spec_verify_trees_greedy(logits, parent, drafted)
        _, ctx = lib.spec_cache_commit(cache, table, ctx, parent, drafted, path, length)
        for b, n in enumerate(length.tolist()):
            out[b] += path[b, :n].tolist()
        last = path.gather(1, (length - 1).long()[:, None])[:, 0].contiguous()
    status = lib.spec_get_status()
    if status:
        raise lib.SpecError(status, "tree_step")
    return out


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=8)
    args.add_argument("--batch", type=int, default=4)
    args.add_argument("--nodes", type=int, default=13)
    args.add_argument("--int8", action="store_true")
    a = args.parse_args()
    done = decode(a.steps, a.batch, a.nodes, kind=torch.int8 if a.int8 else torch.float8_e4m3fn)
    for b, row in enumerate(done):
        print(f"sequence {b}: {len(row)} tokens in {a.steps + 1} passes: {row[:12]}{' ...' if len(row) > 12 else ''}")
