"""Plain 64-bit restatements of the operators from a prompt to a cache within a budget, for the tests, from the
definitions in include/spec_verify.h; they share no code with the kernels or the binding."""
from __future__ import annotations

import math

import torch

from cache_reference import HALF_STEP


def prompt_attention(q, k, v, starts, scale):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits; q [T, Hq, D], k and v [T, Hk, D] on any device."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    half = HALF_STEP[q.dtype]
    for lo, hi in zip(starts, starts[1:]):
        L = hi - lo
        if L == 0:
            continue
        later = torch.ones((L, L), dtype=torch.bool, device=q.device).triu(1)
        for h in range(Hq):
            qq, kk, vv = q[lo:hi, h].double(), k[lo:hi, h // G].double(), v[lo:hi, h // G].double()
            s = (qq @ kk.T * scale).masked_fill(later, -math.inf)
            size = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(later, 0)
            z = torch.logsumexp(s, -1)
            p = (s - z[:, None]).exp()
            # a score is a sum of D products in 32 bits and a few roundings of the result; exponents of up to a few
            # hundred are held in 32 bits, and the exponential's own error is below 2^-20
            off = (D + 8) * 2.0 ** -24 * size.amax(-1) + 2.0 ** -16
            # weights are rounded once to the inputs' type, the output once more; fp16 has a least step, half of which
            # is 2^-25 where the row's largest weight is at least 2^8
            spread = p @ vv.abs()
            least = 0.0
            if q.dtype == torch.float16:
                least = 2.0 ** -33 * p.amax(-1)[:, None] * ((~later).double() @ vv.abs())
            out[lo:hi, h] = p @ vv
            lse[lo:hi, h] = z
            tol[lo:hi, h] = (half + 2 * off[:, None]) * spread + least
            tol_lse[lo:hi, h] = off + 1e-6 * z.abs()
    return out, lse, tol + half * out.abs() * 1.01 + half * tol, tol_lse


def rotate(x, weight, positions, axis, inv_freq, rot, pairs, norm, eps):
    """x [B, N, H, D] in 64 bits; positions [B, N, axes] whole numbers, base included."""
    y = x.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double()
    out = y.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        f = (positions[..., int(axis[i])].double() * float(inv_freq[i]))[..., None]
        out[..., a] = y[..., a] * f.cos() - y[..., b] * f.sin()
        out[..., b] = y[..., b] * f.cos() + y[..., a] * f.sin()
    return out


def slot_weights(cache, b, ctx, cnt, q, lse, mask, scale):
    """One sequence: (sums [Hk, ctx + cnt], their tolerance); q [N, Hq, D] and lse [N, Hq] in 64 bits, mask [N, N] bool or None."""
    N, Hq, D = q.shape
    k = cache.rows(0, b, 0, ctx + cnt)
    H = k.shape[1]
    seen = torch.zeros((N, ctx + cnt), dtype=torch.bool)
    seen[:, :ctx] = True
    node = torch.arange(cnt)
    seen[:, ctx:] = (node[None] <= torch.arange(N)[:, None]) if mask is None else mask[:, :cnt]
    seen[cnt:] = False
    kk = k.repeat_interleave(Hq // H, 1)
    s = torch.einsum("nhd,thd->nht", q, kk) * scale
    # a score: D products in 32 bits; queries below 2^-14 of their row's largest element are off by 2^-25 of it; score
    # times factor minus lse in 32 bits, and the exponential
    size = torch.einsum("nhd,thd->nht", q.abs(), kk.abs()) * abs(scale)
    least = 2.0 ** -25 * q.abs().amax(-1)[..., None] * kk.abs().sum(-1).T[None] * abs(scale)
    off = (D + 8) * 2.0 ** -24 * size + least + 2.0 ** -22 * (s.abs() + lse.abs().nan_to_num(0, 0, 0)[..., None]) + 2.0 ** -20
    live = seen[:, None] & torch.isfinite(lse)[..., None]
    w = torch.where(live, (s - lse[..., None]).exp(), 0.0)
    rows = N * Hq // H
    by_head = lambda x: x.reshape(N, H, Hq // H, -1).sum((0, 2))  # noqa: E731
    return by_head(w), by_head(w * 2 * off) + (rows + 8) * 2.0 ** -24 * by_head(w)


def keeps(weights, ctx, keep, first, last):
    """The slots that one head keeps: its weights as a list of numbers."""
    if ctx <= keep:
        return list(range(ctx))
    free = sorted(range(first, ctx - last), key=lambda s: (math.isnan(weights[s]), 0.0 if math.isnan(weights[s]) else -weights[s], s))
    return sorted(list(range(first)) + free[:keep - first - last] + list(range(ctx - last, ctx)))
