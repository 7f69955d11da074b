"""Plain 64-bit restatements of the cache operators for the tests, on the CPU, one sequence at a time, from the
definitions in include/spec_verify.h; they share no code with the kernels or the binding."""
from __future__ import annotations

import math

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
_E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)


def values(codes, kind):
    """Codes as 64-bit numbers."""
    return _E4M3[codes.view(torch.uint8).long()] if kind == "e4m3" else codes.to(torch.float64)


def nearest(x, kind):
    """64-bit numbers in the codes' range as codes: nearest, ties to even."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127).to(torch.int8)
    grid = _E4M3[:127]                         # the non-negative finite values, ascending; even codes are even
    a = x.abs().clamp(max=448.0).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    take = torch.where(down < up, lo, torch.where(up < down, hi, torch.where(lo % 2 == 0, lo, hi)))
    take = torch.where(grid[hi] == a, hi, take)
    sign = torch.where(torch.signbit(x), 128, 0)
    return (take + sign).to(torch.uint8).view(torch.float8_e4m3fn)


def scale_for(amax, kind):
    e = -100
    while amax > QMAX[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """A cache's state on the CPU."""

    def __init__(self, k, v, ks, vs, table, kind):
        self.codes, self.scales, self.table, self.kind = [k.clone(), v.clone()], [ks.clone(), vs.clone()], table, kind
        self.page = k.shape[2]

    def row(self, t, b, slot):
        p = int(self.table[b, slot // self.page])
        return values(self.codes[t][p, :, slot % self.page], self.kind) * self.scales[t][p].double()[:, None]

    def rows(self, t, b, first, last, scaled=True):
        """[slots, Hk, D]; scaled=False: codes, and the scale of each slot [slots, Hk]."""
        H, D = self.codes[t].shape[1], self.codes[t].shape[3]
        if last <= first:
            empty = torch.zeros((0, H, D), dtype=torch.float64)
            return empty if scaled else (empty, empty[..., 0])
        pages = self.table[b, first // self.page:(last - 1) // self.page + 1].long()
        x = values(self.codes[t].view(torch.uint8)[pages].view(CODE[self.kind]), self.kind)
        scale = self.scales[t][pages].double()[:, :, None, None]
        off = first - first // self.page * self.page
        part = lambda y: y.permute(0, 2, 1, 3).reshape(-1, H, y.shape[-1])[off:off + last - first]  # noqa: E731
        return part(x * scale) if scaled else (part(x), part(scale.expand(-1, -1, self.page, 1))[..., 0])

    def row_f32(self, t, b, slot):
        """As row, the product rounded to 32 bits."""
        p = int(self.table[b, slot // self.page])
        return values(self.codes[t][p, :, slot % self.page], self.kind).float() * self.scales[t][p][:, None]

    def put_f32(self, t, b, start, rows):
        """As put of a commit, for any scales and rows: quotients and products rounded to 32 bits, NaN as 0."""
        code = lambda x: nearest(x.nan_to_num(0.0, math.inf, -math.inf).double(), self.kind).view(torch.uint8)  # noqa: E731
        at = 0
        while at < len(rows):
            blk, r = divmod(start + at, self.page)
            n = min(self.page - r, len(rows) - at)
            p = int(self.table[b, blk])
            for h in range(rows.shape[1]):
                x, old, codes = rows[at:at + n, h], self.scales[t][p, h].clone(), self.codes[t][p, h].view(torch.uint8)
                fine = x[torch.isfinite(x)]
                new = torch.tensor(max(scale_for(fine.abs().max().item() if fine.numel() else 0.0, self.kind), old.item()))
                if new > old:
                    codes.copy_(code(values(self.codes[t][p, h], self.kind).float() * (old / new)))
                    self.scales[t][p, h] = new
                codes[r:r + n] = code(x / new)
            at += n

    def put(self, t, b, start, rows, may_start_anew):
        at = 0
        while at < len(rows):
            blk, r = divmod(start + at, self.page)
            n = min(self.page - r, len(rows) - at)
            p = int(self.table[b, blk])
            for h in range(rows.shape[1]):
                x = rows[at:at + n, h]
                fine = x[torch.isfinite(x)]
                need = scale_for(fine.abs().max().item() if fine.numel() else 0.0, self.kind)
                old = self.scales[t][p, h].item()
                if r or not may_start_anew:
                    new = max(need, old)
                    if new > old:
                        # ratio and product are rounded to 32 bits; exact for powers of two
                        moved = (values(self.codes[t][p, h], self.kind).float() * (torch.tensor(old) / torch.tensor(new))).double()
                        self.codes[t][p, h].view(torch.uint8).copy_(nearest(moved, self.kind).view(torch.uint8))
                else:
                    new = need
                self.scales[t][p, h] = new
                x = torch.where(torch.isnan(x), 0.0, x.clamp(-3e38, 3e38))
                y = (x / new).clamp(-QMAX[self.kind], QMAX[self.kind])
                self.codes[t][p, h, r:r + n].view(torch.uint8).copy_(nearest(y, self.kind).view(torch.uint8))
            at += n


def attention(cache, b, ctx, cnt, q, mask, scale):
    """One sequence: (out, lse, tolerance of out, tolerance of lse), q [N, Hq, D] in 64 bits, mask [N, N] bool or None."""
    N, Hq, D = q.shape
    k, v = (cache.rows(t, b, 0, ctx + cnt) for t in (0, 1))
    H = k.shape[1]
    seen = torch.zeros((N, ctx + cnt), dtype=torch.bool)
    seen[:, :ctx] = True
    node = torch.arange(cnt)
    seen[:, ctx:] = (node[None] <= torch.arange(N)[:, None]) if mask is None else mask[:, :cnt]
    seen[cnt:] = False
    kk = k.repeat_interleave(Hq // H, 1)
    vv = v.repeat_interleave(Hq // H, 1)
    s = torch.einsum("nhd,thd->nht", q, kk) * scale
    size = torch.einsum("nhd,thd->nht", q.abs(), kk.abs()) * abs(scale)
    s = s.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1) if ctx + cnt else torch.full((N, Hq), -math.inf, dtype=torch.float64)
    p = torch.where(seen[:, None], (s - lse[..., None].clamp(min=-1e300)).exp(), 0.0)
    out = torch.einsum("nht,thd->nhd", p, vv)
    # a score is a sum of D products in 32 bits and a few roundings of the result; a weight is rounded to fp16 once
    # (half a step 2^-11), and exponents of up to a few hundred are held in 32 bits
    off = torch.where(seen[:, None], (D + 8) * 2.0 ** -24 * size, 0.0)
    off = (off.amax(-1) if off.shape[-1] else torch.zeros((N, Hq), dtype=torch.float64)) + 2.0 ** -16
    spread = torch.einsum("nht,thd->nhd", p, vv.abs())
    # below 2^-27 of the row's largest weight (weights times value scales) fp16 has a least step instead: half of it is
    # 2^-25 where the largest weight is at least 2^13
    codes, vs = cache.rows(1, b, 0, ctx + cnt, scaled=False)
    vs = vs.clamp(min=2.0 ** -100).repeat_interleave(Hq // H, 1).T
    top = (p * vs[None]).amax(-1) if ctx + cnt else torch.zeros((N, Hq), dtype=torch.float64)
    least = 2.0 ** -38 * top[..., None] * torch.einsum("nt,thd->nhd", seen.double(), codes.abs().repeat_interleave(Hq // H, 1))
    return out, lse, (2.0 ** -11 + 2 * off)[..., None] * spread + least, off + 1e-6 * lse.abs().nan_to_num(0, 0, 0)
