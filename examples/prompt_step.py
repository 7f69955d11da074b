"""From prompts with pictures to decoding within a budget, with the library's calls only for what it does.

One attention layer with random weights stands in for the target model.  Prompts of different lengths, each with a
picture in it, stand packed one behind the other: their queries and keys are turned by positions with three axes, attend
causally, and go into a paged 8-bit cache.  The last tokens of each prompt weigh their context, slots that received
little attention are given up until every context fits its budget, and decoding goes on with draft trees, whose tokens
stand at their true positions whatever the cache still holds.

    python examples/prompt_step.py [--batch 3] [--keep 64] [--steps 4] [--int8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sampling_row_online_gb300 as lib  # noqa: E402
from tree_step import Layer, draft_trees  # noqa: E402


def positions_of(length, wide=6, text=9):
    """[length, 3] and the position that follows: `text` tokens of text, a picture of wide * wide tokens, text again.  A text
    token stands at one position on all axes, a picture's at one time and its row and column."""
    rows = []
    for i in range(length):
        if text <= i < text + wide * wide:
            cell = i - text
            rows.append([text, text + cell // wide, text + cell % wide])
        else:
            at = i if i < text else i - wide * wide + wide
            rows.append([at] * 3)
    return torch.tensor(rows, dtype=torch.int32), max(max(r) for r in rows) + 1


def serve(batch=3, keep=64, steps=4, nodes=13, window=8, first=4, kind=torch.float8_e4m3fn, vocab=4096, page=32, seed=1):
    """Returns (the committed tokens of each sequence, the slots that each kv head kept or None, the last logits of the
    prompts)."""
    layer = Layer(vocab, heads=8, kv_heads=2, dim=128)
    H, D = layer.kv_heads, layer.dim
    g = torch.Generator(device="cuda").manual_seed(seed)
    lengths = [61 + 38 * b for b in range(batch)]
    starts = torch.tensor([sum(lengths[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
    T = sum(lengths)
    tokens = torch.randint(0, vocab, (T,), generator=g, device="cuda")
    where = [positions_of(n) for n in lengths]
    positions = torch.cat([p for p, _ in where]).cuda()[None].contiguous()
    base = torch.tensor([after for _, after in where], dtype=torch.int32, device="cuda")  # of the next token
    axis = (torch.arange(D // 2) % 3).to(torch.int32)

    # the prompts' pass
    x = layer.embed[tokens]
    q, k, v = ((x @ w).view(1, T, -1, D) for w in (layer.wq, layer.wk, layer.wv))
    q, k = lib.spec_qk_norm_rope_axes(q, k, layer.inv_freq, axis, positions, q_weight=layer.q_norm, k_weight=layer.k_norm)
    out, _ = lib.spec_prompt_attention(q[0], k[0], v[0], starts)
    ends = starts[1:].long() - 1
    logits = (x[ends] + out[ends].view(batch, -1)) @ layer.head
    last = logits.argmax(-1).to(torch.int32)

    # into the cache, each sequence's rows as they lie
    per = -(-(max(lengths) + (steps + 1) * nodes) // page)
    cache = lib.SpecCache.empty(batch * per, H, page, D, dtype=kind)
    table = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32).view(batch, per)
    zero = torch.zeros((1,), dtype=torch.int32, device="cuda")
    for b, (lo, hi) in enumerate(zip(starts.tolist(), starts.tolist()[1:])):
        lib.spec_cache_write(cache, table[b:b + 1], zero, k[:, lo:hi], v[:, lo:hi])
    ctx = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    # the prompts' last tokens weigh their contexts, and what received little goes
    kept = None
    weights = torch.zeros((batch, H, per * page), device="cuda")
    if keep is not None:
        rows = ends[:, None] - window + 1 + torch.arange(window, device="cuda")
        before = ctx - window
        asked = q[0, rows]
        _, lse = lib.spec_cache_attention(asked, cache, table, before, want_lse=True)
        lib.spec_cache_weights(asked, cache, table, before, lse, weights)
        kept, ctx = lib.spec_cache_evict(cache, table, ctx, weights, keep, first=first, last=window)

    # decoding
    done = [[int(t)] for t in last]
    for step in range(steps):
        parent, drafted = draft_trees(layer, last, nodes, seed * 1000 + step)
        mask, depth = lib.spec_tree_mask(parent)
        x = layer.embed[drafted.long()]
        q, k, v = ((x @ w).view(batch, nodes, -1, D) for w in (layer.wq, layer.wk, layer.wv))
        q, k = lib.spec_qk_norm_rope(q, k, layer.inv_freq, base=base, offset=depth, q_weight=layer.q_norm, k_weight=layer.k_norm)
        lib.spec_cache_write(cache, table, ctx, k, v)
        out, _ = lib.spec_cache_attention(q, cache, table, ctx, mask=mask)
        logits_t = (x + out.view(batch, nodes, -1)) @ layer.head
        path, length = lib.spec_verify_trees_greedy(logits_t, parent, drafted)
        _, ctx = lib.spec_cache_commit(cache, table, ctx, parent, drafted, path, length)
        base = base + length
        for b, n in enumerate(length.tolist()):
            done[b] += path[b, :n].tolist()
        last = path.gather(1, (length - 1).long()[:, None])[:, 0].contiguous()
    status = lib.spec_get_status()
    if status:
        raise lib.SpecError(status, "prompt_step")
    return done, kept, logits


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--batch", type=int, default=3)
    args.add_argument("--keep", type=int, default=64)
    args.add_argument("--steps", type=int, default=4)
    args.add_argument("--int8", action="store_true")
    a = args.parse_args()
    done, kept, _ = serve(a.batch, a.keep, a.steps, kind=torch.int8 if a.int8 else torch.float8_e4m3fn)
    for b, row in enumerate(done):
        print(f"sequence {b}: kv head 0 kept slots {kept[b, 0, :6].tolist()} ...; {len(row)} tokens: {row[:10]}{' ...' if len(row) > 10 else ''}")
