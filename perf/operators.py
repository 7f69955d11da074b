"""The operators of a speculative step around an 8-bit paged key/value cache: their cases, inputs and plain forms.

One layer of the target model verifies a chain or a tree of drafted tokens in five calls: the queries' and keys'
norms with the rotation (positions are the context length plus the node's depth), the quantised write of the nodes'
keys and values behind the context, the attention over the cache under the tree's mask, and, once the verification
has chosen a path, the commit that moves the accepted nodes' rows together.  The fifth reads a cache back.

The cache holds codes of 8 bits (e4m3, or int8) in pages [pages, kv_heads, page_size, head_dim] and one scale for
each page and head: a block's values are code * scale.  The scales that the write and the commit give are powers of
two, the least with amax <= qmax * scale (qmax: 448 for e4m3, 127 for int8), at least 2^-100.
"""
import math

import torch

own = False

E4M3, I8 = "e4m3", "int8"
QMAX = {E4M3: 448.0, I8: 127.0}
CODE = {E4M3: torch.float8_e4m3fn, I8: torch.int8}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # 64 sequences verify 5 drafts and the root: 6 tokens each go through the norms and the rotation
        dict(name="rope_chain", op="rope", B=64, N=6, Hq=32, Hk=8, D=128, dtype="bf16", rot=128, pairs=False,
             norm=True, tree=False, theta=1e6),
        # a prompt's pass: 4 sequences of 4095 tokens, half of each head rotated in neighbouring pairs
        dict(name="rope_prompt", op="rope", B=4, N=4095, Hq=32, Hk=8, D=128, dtype="bf16", rot=64, pairs=True,
             norm=True, tree=False, theta=1e4),
        # a decoding step of 64 sequences: one new token each into pages that are partly filled
        dict(name="write_step", op="write", B=64, N=1, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=4096, ragged=False),
        # a prompt's keys and values, 8 sequences of up to 8000 tokens, into an int8 cache
        dict(name="write_prompt", op="write", B=8, N=8000, Hk=8, D=128, page=64, dtype="bf16", kind=I8, L=1000, ragged=True),
        # one sequence's short context is handed on in 32 bits
        dict(name="read_short", op="read", B=1, N=513, Hk=8, D=64, page=16, dtype="f32", kind=I8, ragged=False),
        # contexts of up to 32768 tokens are read back in bf16, as to move a session or to run another attention
        dict(name="read_long", op="read", B=8, N=32768, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, ragged=True),
        # the paths that 32 trees of 63 nodes accepted
        dict(name="commit_tree", op="commit", B=32, N=63, Hk=8, D=128, page=64, kind=E4M3, L=4096, depth=4),
        # a large batch of deep trees
        dict(name="commit_batch", op="commit", B=256, N=255, Hk=8, D=128, page=32, kind=I8, L=1000, depth=30),
        # one sequence decodes one token: the latency of a single user's step
        dict(name="attend_one", op="attend", B=1, N=1, Hq=32, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=4096,
             mask="chain", ragged=False),
        # a batch that decodes one token over long contexts
        dict(name="attend_long", op="attend", B=64, N=1, Hq=64, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=32768,
             mask="chain", ragged=True),
        # 64 sequences verify chains of 5 drafts over an int8 cache
        dict(name="attend_chain", op="attend", B=64, N=6, Hq=32, Hk=8, D=128, page=32, dtype="bf16", kind=I8, L=8192,
             mask="chain", ragged=True),
        # 32 trees of 63 nodes over long contexts
        dict(name="attend_tree", op="attend", B=32, N=63, Hq=32, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=16384,
             mask="tree", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "commit", "attend", "attend", "attend"])
    kind, page, D = rng.choice([E4M3, I8]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rope":
        N = _log(rng, 1, 4095)
        B = _log(rng, 1, max(1, min(256, 16380 // N)))
        Dr = rng.choice([64, 80, 128, 128, 256])
        H = rng.choice([1, 2, 4, 8])
        return dict(op=op, B=B, N=N, Hq=H * rng.choice([1, 3, 4]) if Dr <= 128 else H * 2, Hk=H, D=Dr,
                    dtype=rng.choice(["bf16", "f16", "f32"]) if N * B < 4000 else "bf16",
                    rot=rng.choice([Dr, Dr // 2, Dr // 4 * 2]), pairs=rng.random() < 0.4, norm=rng.random() < 0.8,
                    tree=N <= 255 and rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 1e6]))
    if op == "write":
        N = _log(rng, 1, 8000)
        B = _log(rng, 1, max(1, min(256, 64000 // N)))
        return dict(op=op, B=B, N=N, Hk=Hk, D=D, page=page, dtype=rng.choice(["bf16", "f16", "f32"]) if N * B < 16000 else "bf16",
                    kind=kind, L=_log(rng, 1, 4096), ragged=rng.random() < 0.5)
    if op == "read":
        N = _log(rng, 1, 32768)
        B = _log(rng, 1, max(1, min(256, 8 * 32768 // N)))
        return dict(op=op, B=B, N=N, Hk=Hk, D=D, page=page, dtype=rng.choice(["bf16", "f16", "f32"]) if N * B < 65536 else "bf16",
                    kind=kind, ragged=rng.random() < 0.5)
    if op == "commit":
        N = _log(rng, 12, 255)
        return dict(op=op, B=_log(rng, 1, 256), N=N, Hk=Hk, D=D, page=page, kind=kind, L=_log(rng, 1, 4096),
                    depth=rng.randint(1, max(1, min(30, N // 8))))
    shape = rng.choice(["one", "chain", "tree", "part"])
    N = {"one": 1, "chain": rng.randint(2, 9), "tree": rng.randint(10, 64), "part": _log(rng, 65, 1024)}[shape]
    L = _log(rng, 1, 32768)
    most = min(256, int(64 * 32768 * 8 // ((L + N) * Hk)), int(4e8 // (N * Hk * G * (L + N))) + 1)
    return dict(op=op, B=_log(rng, 1, max(1, most)), N=N, Hq=Hk * G, Hk=Hk, D=D, page=page, dtype=rng.choice(["bf16", "bf16", "f16"]),
                kind=kind, L=L, mask="tree" if shape == "tree" or N <= 255 and rng.random() < 0.3 else "chain",
                ragged=rng.random() < 0.7)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * SIZE[c["dtype"]], "flops": 8 * n}
    tokens, rows = _expected(c)
    elems = 2 * c["Hk"] * c["D"]
    if c["op"] == "write":
        return {"bytes": rows * elems * (SIZE[c["dtype"]] + 1), "flops": 3 * rows * elems}
    if c["op"] == "read":
        return {"bytes": rows * elems * (SIZE[c["dtype"]] + 1), "flops": rows * elems}
    if c["op"] == "commit":
        return {"bytes": 2 * rows * elems + 4 * c["B"] * 2 * c["N"], "flops": 3 * rows * elems}
    q = c["B"] * c["N"] * c["Hq"] * c["D"]
    pages = -(-tokens // c["page"])
    return {"bytes": tokens * elems + 8 * pages * c["Hk"] + 2 * q * SIZE[c["dtype"]] + 4 * c["B"] * c["N"] * c["Hq"],
            "flops": 4 * c["N"] * c["Hq"] * c["D"] * tokens}


def _expected(c):
    """(tokens that all sequences hold together, rows that the call handles), on average over the seeds."""
    part = 0.75 if c.get("ragged") else 1.0
    if c["op"] == "read":
        return int(c["B"] * c["N"] * part), int(c["B"] * c["N"] * part)
    if c["op"] == "write":
        return int(c["B"] * (c["L"] + c["N"])), int(c["B"] * c["N"] * part)
    if c["op"] == "commit":
        return c["B"] * (c["L"] + c["N"]), int(c["B"] * (1 + c["depth"] / 2))
    return int(c["B"] * (c["L"] * part + c["N"])), c["B"] * c["N"]


# ----------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _whole(g, lo, hi, shape):
    """Whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _pages(g, c, most):
    """A pool, and a table that gives every sequence its own pages in a mixed order; entries past `most` tokens do not exist."""
    per = -(-most // c["page"])
    table = torch.randperm(c["B"] * per, generator=g, device="cuda").to(torch.int32).reshape(c["B"], per)
    return c["B"] * per, table.contiguous()


def _cache(g, c, pages):
    """Codes and scales as the write gives them for normal values whose size differs between heads and, by a factor of two, between blocks."""
    shape = (pages, c["Hk"], c["page"], c["D"])
    cache = {}
    for name in ("k", "v"):
        codes = torch.empty(shape, dtype=CODE[c["kind"]], device="cuda")
        for at in range(0, pages, 4096):
            part = torch.randn((min(4096, pages - at),) + shape[1:], generator=g, device="cuda")
            part = part.mul_(QMAX[c["kind"]] / 5).clamp_(-QMAX[c["kind"]], QMAX[c["kind"]])
            codes[at:at + 4096] = part.round_() if c["kind"] == I8 else part
        # sizes of about 1/2 to 2 of a value: a fifth of the largest code times the scale
        power = _whole(g, 0, 1, (pages, c["Hk"])) + _whole(g, -1, 0, (1, c["Hk"])) + round(math.log2(5 / QMAX[c["kind"]]))
        cache[name], cache[name + "_scale"] = codes, _two_to(power)
    return cache


def _tree(g, c, depth):
    """Trees listed level by level, the parents of a level in the one above it: parent [B, N] and the depth of each node.
    The first level has at least as many nodes as there are levels."""
    B, N = c["B"], c["N"]
    first = [0, 1] + [1 + depth + (N - 1 - depth) * d // depth for d in range(1, depth)] + [N] if depth else [0, N]
    parent = torch.empty((B, N), dtype=torch.int32, device="cuda")
    level = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    parent[:, 0] = -1
    for d in range(1, len(first) - 1):
        lo, mid, hi = first[d - 1], first[d], first[d + 1]
        parent[:, mid:hi] = _whole(g, lo, mid - 1, (B, hi - mid))
        parent[:, mid] = lo
        level[:, mid:hi] = d
    return parent, level


def _ancestors(parent, depth):
    """[B, N, N]: whether node j is on the path of node i."""
    B, N = parent.shape
    seen = torch.eye(N, dtype=torch.bool, device="cuda").expand(B, N, N).clone()
    at = parent.long()
    for _ in range(depth):
        seen |= torch.zeros_like(seen).scatter_(2, at.clamp(min=0)[..., None], (at >= 0)[..., None])
        at = torch.where(at >= 0, parent.long().gather(1, at.clamp(min=0)), at)
    return seen


def _words(seen):
    """The bits of [B, N, N] in words of 32, [B, N, ceil(N / 32)] int32."""
    B, N, _ = seen.shape
    W = -(-N // 32)
    bits = torch.zeros((B, N, W * 32), dtype=torch.int64, device="cuda")
    bits[..., :N] = seen
    words = (bits.reshape(B, N, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _lengths(g, c, most):
    return _whole(g, -(-most // 2), most, (c["B"],)) if c.get("ragged") else torch.full((c["B"],), most, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}
    B, N = c["B"], c["N"]
    if c["op"] == "rope":
        t = DTYPE[c["dtype"]]
        s["q"] = torch.randn((B, N, c["Hq"], c["D"]), generator=g, device="cuda").mul_(2).to(t)
        s["k"] = torch.randn((B, N, c["Hk"], c["D"]), generator=g, device="cuda").mul_(2).to(t)
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(c["D"], generator=g, device="cuda")).to(t) if c["norm"] else None
        s["base"] = _whole(g, 0, 130000, (B,))
        s["offset"] = _tree(g, c, max(1, min(5, N // 8)))[1] if c["tree"] and N > 1 else None
        half = torch.arange(c["rot"] // 2, dtype=torch.float64)
        s["inv_freq"] = c["theta"] ** (-2 * half / c["rot"])
        return s
    if c["op"] == "read":
        pages, s["table"] = _pages(g, c, N)
        s |= _cache(g, c, pages)
        s["start"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
        s["counts"] = _lengths(g, c, N)
        return s
    L = c["L"]
    pages, s["table"] = _pages(g, c, L + N)
    s |= _cache(g, c, pages)
    if c["op"] == "write":
        t = DTYPE[c["dtype"]]
        for name in ("k_new", "v_new"):
            s[name] = torch.randn((B, N, c["Hk"], c["D"]), generator=g, device="cuda").mul_(2).to(t)
        s["ctx"] = _whole(g, L // 2, L, (B,))
        s["counts"] = _lengths(g, c, N)
        return s
    if c["op"] == "commit":
        s["ctx"] = _whole(g, L // 2, L, (B,))
        s["parent"], level = _tree(g, c, c["depth"])
        s["tokens"] = _whole(g, 0, 32767, (B, N))
        # a path from the root through its first child (the most probable one) downwards, as long as the tree has nodes for it
        path = torch.full((B, c["depth"] + 1), -1, dtype=torch.int32, device="cuda")
        length = torch.ones((B,), dtype=torch.int32, device="cuda")
        at = torch.zeros((B,), dtype=torch.int64, device="cuda")
        most = _whole(g, 0, c["depth"], (B,))
        open_ = torch.ones((B,), dtype=torch.bool, device="cuda")
        for d in range(c["depth"]):
            child = (s["parent"] == at[:, None]) & (level == d + 1)
            pick = child.float() * (torch.rand((B, N), generator=g, device="cuda") + 0.01)
            best = pick.argmax(1) if d else torch.ones_like(at)
            open_ = open_ & child.any(1) & (most > d)
            at = torch.where(open_, best, at)
            path[:, d] = torch.where(open_, s["tokens"].gather(1, at[:, None])[:, 0], -1)
            length += open_.to(torch.int32)
        bonus = _whole(g, 0, 32767, (B, 1))
        s["path"] = path.scatter(1, (length - 1)[:, None].long(), bonus).contiguous()
        s["length"] = length
        return s
    s["ctx"] = _lengths(g, c, L)
    s["q"] = torch.randn((B, N, c["Hq"], c["D"]), generator=g, device="cuda").mul_(1.5).to(DTYPE[c["dtype"]])
    depth = max(1, min(5, N // 8)) if N > 1 else 0
    s["mask"] = _words(_ancestors(_tree(g, c, depth)[0], depth)) if c["mask"] == "tree" else None
    return s


# ------------------------------------------------------------------- runs
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import sampling_row_online_gb300 as lib
        if op == "rope":
            return lib.spec_qk_norm_rope(s["q"], s["k"], s["inv_freq"], base=s["base"], offset=s["offset"], norm=s["case"]["norm"],
                                         q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6, pairs=s["case"]["pairs"])
        cache = lib.SpecCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "read":
            return lib.spec_cache_read(cache, s["table"], s["start"], s["counts"], s["case"]["N"],
                                       dtype=DTYPE[s["case"]["dtype"]])
        if op == "write":
            lib.spec_cache_write(cache, s["table"], s["ctx"], s["k_new"], s["v_new"], counts=s["counts"])
            return s["k"], s["v"], s["k_scale"], s["v_scale"]
        if op == "commit":
            index, length = lib.spec_cache_commit(cache, s["table"], s["ctx"], s["parent"], s["tokens"], s["path"], s["length"])
            return index, length, s["k"], s["v"], s["k_scale"], s["v_scale"]
        return lib.spec_cache_attention(s["q"], cache, s["table"], s["ctx"], mask=s["mask"], want_lse=True)
    return {"rope": _rope, "read": _read, "write": _write, "commit": _commit, "attend": _attend}[op](s)


def _rope(s):
    c = s["case"]
    B, N = c["B"], c["N"]
    index = torch.arange(N, device="cuda", dtype=torch.int32)[None] if s["offset"] is None else s["offset"]
    angle = (s["base"][:, None] + index).double()[..., None] * s["inv_freq"].to("cuda")
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, weight):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r = c["rot"]
        out = y.clone()
        a, b = (slice(0, r, 2), slice(1, r, 2)) if c["pairs"] else (slice(0, r // 2), slice(r // 2, r))
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
        return out.to(x.dtype)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


def _gathered(s, name, dtype=torch.float32):
    """[B, Hk, slots, D]: the values of each sequence's pages in order."""
    c = s["case"]
    table = s["table"].long()
    values = s[name][table].to(dtype) * s[name + "_scale"][table][..., None, None].to(dtype)
    return values.permute(0, 2, 1, 3, 4).reshape(c["B"], c["Hk"], -1, c["D"])


def _read(s):
    c = s["case"]
    slot = torch.arange(c["N"], device="cuda")
    got = []
    for name in ("k", "v"):
        x = _gathered(s, name)[:, :, :c["N"]].transpose(1, 2)
        got.append(x.masked_fill((slot >= s["counts"][:, None])[..., None, None], 0).to(DTYPE[c["dtype"]]))
    return tuple(got)


def _two_to(power):
    """2^power in 32 bits by its bits (torch's pow and ldexp round on the GPU), for powers from -126 to 127."""
    return (power.to(torch.int32) + 127 << 23).view(torch.float32)


def _scale_for(amax, kind):
    """The least power of two with amax <= qmax * scale, at least 2^-100."""
    half, power = torch.frexp(amax)
    top, up = math.frexp(QMAX[kind])
    power = torch.where(amax > 0, power - up + (half > top).to(power.dtype), -100)
    return _two_to(power.clamp(min=-100))


def _codes(x, kind):
    return x.round().clamp(-127, 127).to(torch.int8) if kind == I8 else x.to(torch.float8_e4m3fn)


def _put(s, name, rows, start, valid, fresh):
    """Puts the `valid` ones of `rows` [B, M, Hk, D] (32 bits) into the slots from `start` [B] on, block by block: a block's scale grows
    to what its new rows need, and what it held is rounded to the new scale; where `fresh`, a block that holds nothing before
    `start` takes the scale of its new rows alone."""
    c = s["case"]
    page, kind, (B, M, Hk, D) = c["page"], c["kind"], rows.shape
    blocks = (M + page - 2) // page + 1  # that M rows can touch
    first = start // page
    block = first[:, None] + torch.arange(blocks, device="cuda")
    pages = s["table"].long().gather(1, block.clamp(max=s["table"].shape[1] - 1))
    at = (start - first * page)[:, None] + torch.arange(M, device="cuda")
    full = torch.zeros((B, blocks * page, Hk, D), device="cuda")
    full.scatter_(1, at[..., None, None].expand(rows.shape), rows.masked_fill(~valid[..., None, None], 0))
    new = torch.zeros((B, blocks * page), dtype=torch.bool, device="cuda").scatter_(1, at, valid)
    full = full.reshape(B, blocks, page, Hk, D).transpose(2, 3)
    new = new.reshape(B, blocks, 1, page, 1)
    need = _scale_for(full.abs().amax((3, 4)), kind)
    old = s[name + "_scale"][pages]
    empty = (block * page >= start[:, None])[..., None] & fresh
    scale = torch.where(empty, need, torch.maximum(need, old))
    codes = s[name].view(torch.uint8)[pages]
    ratio = torch.where(empty, 1, old / scale)[..., None, None]
    held = torch.where(ratio < 1, _codes(codes.view(CODE[kind]).float() * ratio, kind).view(torch.uint8), codes)
    codes = torch.where(new, _codes(full / scale[..., None, None], kind).view(torch.uint8), held)
    b, j = torch.nonzero(new.any(3).reshape(B, blocks), as_tuple=True)
    s[name].view(torch.uint8)[pages[b, j]] = codes[b, j]
    s[name + "_scale"][pages[b, j]] = scale[b, j]


def _write(s):
    index = torch.arange(s["case"]["N"], device="cuda")
    for name in ("k", "v"):
        _put(s, name, s[name + "_new"].float(), s["ctx"].long(), index < s["counts"][:, None], True)
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _accepted(s):
    """[B, depth + 1]: the nodes of the accepted path (of several the deepest one's lowest index), then -1."""
    c = s["case"]
    B, N = c["B"], c["N"]
    parent, tokens, length = s["parent"].long(), s["tokens"], s["length"].long()
    up = parent.clamp(min=0)
    depth = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    fits = torch.zeros((B, N), dtype=torch.bool, device="cuda")
    fits[:, 0] = True
    for d in range(1, c["depth"] + 1):  # nodes of depth d whose path so far is the accepted one's
        on = (depth.gather(1, up) == d - 1) & fits.gather(1, up) & (parent >= 0) & (tokens == s["path"][:, d - 1:d]) & (depth == 0)
        on &= (d < length)[:, None]
        on[:, 0] = False
        depth, fits = torch.where(on, d, depth), fits | on
    last = (fits & (depth == (length - 1)[:, None])).int().argmax(1)
    index = torch.full((B, c["depth"] + 1), -1, dtype=torch.int64, device="cuda")
    for d in range(c["depth"], -1, -1):
        here = d < length
        index[:, d] = torch.where(here, last, -1)
        last = torch.where(here, up.gather(1, last[:, None])[:, 0], last)
    return index


def _commit(s):
    c = s["case"]
    index = _accepted(s)
    at = torch.arange(c["depth"] + 1, device="cuda")
    moved = (index >= 0) & (index != at)
    source = s["ctx"].long()[:, None] + index.clamp(min=0)
    page = s["table"].long().gather(1, source // c["page"])
    for name in ("k", "v"):
        rows = s[name].view(torch.uint8)[page, :, source % c["page"]].view(CODE[c["kind"]]).float() * s[name + "_scale"][page][..., None]
        _put(s, name, rows, s["ctx"].long(), moved, False)
    return index.to(torch.int32), s["ctx"] + s["length"], s["k"], s["v"], s["k_scale"], s["v_scale"]


def _seen(s, slots):
    """[B, N, slots]: which slots each node sees: the context, and the nodes of its mask or, without one, those up to itself."""
    c = s["case"]
    N = c["N"]
    slot = torch.arange(slots, device="cuda")
    node = slot - s["ctx"].long()[:, None]
    if s["mask"] is None:
        nodes = torch.ones((N, N), dtype=torch.bool, device="cuda").tril().expand(c["B"], N, N)
    else:
        nodes = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).reshape(c["B"], N, -1)[..., :N] > 0
    at = node.clamp(0, N - 1)[:, None].expand(c["B"], N, slots)
    return (node < 0)[:, None] | nodes.gather(2, at) & ((node >= 0) & (node < N))[:, None]


def _attend(s):
    c = s["case"]
    B, N, Hk, D = c["B"], c["N"], c["Hk"], c["D"]
    G = c["Hq"] // Hk
    q = s["q"].float().reshape(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    score = q @ _gathered(s, "k").transpose(2, 3) * D ** -0.5
    slots = score.shape[-1]
    score = score.reshape(B, Hk, G, N, slots).masked_fill_(~_seen(s, slots)[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top.clamp(min=-1e30)).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.reshape(B, Hk, G * N, slots) @ _gathered(s, "v")).reshape(B, Hk, G, N, D)
    out = torch.where(total > 0, out / total, 0)
    lse = (top + total.log())[..., 0]
    return (out.permute(0, 3, 1, 2, 4).reshape(B, N, c["Hq"], D).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).reshape(B, N, c["Hq"]).contiguous())


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """In 64 bits and one sequence at a time, from the definitions."""
    c = case
    s = prepare(c, seed)
    return {"rope": _exact_rope, "read": _exact_read, "write": _exact_write, "commit": _exact_commit, "attend": _exact_attend}[c["op"]](s)


def _exact_rope(s):
    c = s["case"]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            y = x[b].double()
            if c["norm"]:
                y = y / (y.square().sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
            where = s["base"][b].item() + (torch.arange(c["N"], device="cuda") if s["offset"] is None else s["offset"][b])
            z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), where.double()[:, None] * s["inv_freq"].cuda())[:, None]
            r = c["rot"]
            turned = y[..., :r].unflatten(-1, (r // 2, 2) if c["pairs"] else (2, r // 2))
            turned = turned if c["pairs"] else turned.transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(turned.contiguous()) * z)
            turned = turned if c["pairs"] else turned.transpose(-1, -2)
            out[b] = torch.cat([turned.flatten(-2), y[..., r:]], -1)
        got.append(out)
    return tuple(got)


def _values_of(s, name, b, first, last):
    """[last - first, Hk, D] in 64 bits: the values in slots [first, last) of sequence b."""
    c = s["case"]
    lo = first // c["page"]
    pages = s["table"][b, lo:-(-last // c["page"])].long()
    x = s[name].view(torch.uint8)[pages].view(CODE[c["kind"]]).double() * s[name + "_scale"][pages].double()[..., None, None]
    return x.transpose(1, 2).reshape(-1, c["Hk"], c["D"])[first - lo * c["page"]:last - lo * c["page"]]


def _exact_read(s):
    c = s["case"]
    got = []
    for name in ("k", "v"):
        out = torch.zeros((c["B"], c["N"], c["Hk"], c["D"]), dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["counts"].tolist()):
            out[b, :n] = _values_of(s, name, b, 0, n)
        got.append(out)
    return tuple(got)


def _exact_scale(amax, kind):
    """The least power of two from 2^-100 with amax <= qmax * 2^e: all candidates are tried."""
    all_ = torch.tensor([2.0 ** e for e in range(-100, 128)], dtype=torch.float64, device="cuda")
    return all_[torch.searchsorted(all_ * QMAX[kind], amax)]


def _exact_rounding(x, kind):
    """x (64 bits, within the codes' range) to the nearest code value, ties to even: the spacing is 1, or that of e4m3 at x."""
    if kind == I8:
        return torch.round(x)
    at = torch.tensor([2.0 ** e for e in range(-6, 9)], dtype=torch.float64, device="cuda")
    step = at[torch.searchsorted(at, x.abs(), right=True).clamp(min=1) - 1] / 8
    return torch.round(x / step) * step


def _exact_put(s, b, start, rows, fresh):
    """Sequence b's blocks from `start` on take `rows` (two of [n, Hk, D], 64 bits): code values as 64-bit numbers."""
    c = s["case"]
    for name, x in zip(("k", "v"), rows):
        at = 0
        while at < len(x):
            block = (start + at) // c["page"]
            row = (start + at) % c["page"]
            n = min(c["page"] - row, len(x) - at)
            page = s["table"][b, block].item()
            part = x[at:at + n].transpose(0, 1)
            scale = _exact_scale(part.abs().amax((1, 2)), c["kind"])
            if row or not fresh:
                old = s["exact"][name + "_scale"][page].clone()
                scale = torch.maximum(scale, old)
                grown = _exact_rounding(s["exact"][name][page] * (old / scale)[:, None, None], c["kind"])
                s["exact"][name][page] = torch.where((scale > old)[:, None, None], grown, s["exact"][name][page])
            s["exact"][name][page, :, row:row + n] = _exact_rounding(part / scale[:, None, None], c["kind"])
            s["exact"][name + "_scale"][page] = scale
            at += n


def _exact_state(s):
    big = s["k"].numel() > 4e8
    s["exact"] = None if big else {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    return not big


def _exact_kept(s):
    """The codes as the values they stand for (whole numbers have no 64-bit value to be compared with), and the scales."""
    whole = s["case"]["kind"] == I8
    return tuple(None if whole and n in ("k", "v") else s["exact"][n] for n in ("k", "v", "k_scale", "v_scale"))


def _exact_write(s):
    c = s["case"]
    if not _exact_state(s) or c["B"] * (c["N"] // c["page"] + 2) > 6000:
        return None
    for b, n in enumerate(s["counts"].tolist()):
        _exact_put(s, b, s["ctx"][b].item(), [s[x][b, :n].double() for x in ("k_new", "v_new")], True)
    return _exact_kept(s)


def _exact_commit(s):
    c = s["case"]
    if not _exact_state(s):
        return None
    for b in range(c["B"]):
        parent, tokens, ctx = s["parent"][b].tolist(), s["tokens"][b].tolist(), s["ctx"][b].item()
        want = s["path"][b, :s["length"][b].item() - 1].tolist()
        for node in range(c["N"]):
            path, at = [], node
            while at >= 0:
                path.insert(0, at)
                at = parent[at]
            if [tokens[i] for i in path[1:]] == want:
                break
        first = next((i for i, n in enumerate(path) if i != n), len(path))
        rows = [torch.cat([_values_of(s, x, b, ctx + n, ctx + n + 1) for n in path[first:]] or [torch.zeros((0, c["Hk"], c["D"]), device="cuda")]).double()
                for x in ("k", "v")]
        _exact_put(s, b, ctx + first, rows, False)
    return (None, None) + _exact_kept(s)


def _exact_attend(s):
    c = s["case"]
    B, N, Hk, D = c["B"], c["N"], c["Hk"], c["D"]
    G = c["Hq"] // Hk
    if work(c)["flops"] > 1.2e12:
        return None
    out = torch.zeros((B, N, c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["ctx"].tolist()):
        k, v = (_values_of(s, name, b, 0, L + N).transpose(0, 1) for name in ("k", "v"))
        sees = torch.ones((N, L + N), dtype=torch.bool, device="cuda")
        node = torch.arange(N, device="cuda")
        sees[:, L:] = node[None] <= node[:, None] if s["mask"] is None else (s["mask"][b][:, node // 32] >> (node % 32).int() & 1).bool()
        q = s["q"][b].double().reshape(N, Hk, G, D).permute(1, 2, 0, 3)
        score = torch.einsum("hgnd,htd->hgnt", q, k) / math.sqrt(D)
        score = score.masked_fill(~sees, -math.inf)
        each = torch.logsumexp(score, -1)
        weight = (score - each[..., None]).exp()
        out[b] = torch.einsum("hgnt,htd->hgnd", weight, v).permute(2, 0, 1, 3).reshape(N, c["Hq"], D)
        lse[b] = each.permute(2, 0, 1).reshape(N, c["Hq"])
    return out, lse
