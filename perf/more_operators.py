"""From a prompt to a cache within a budget: the operators' cases, inputs and plain forms.

A prompt's pass through one layer turns its queries and keys by positions that may have several axes (time, height and
width of an image's or a video's tokens), attends causally among the tokens of each of several sequences that stand
packed one behind the other, and, once keys and values are in the paged 8-bit cache, adds up how much attention each
cached slot has received; where a context is longer than the budget allows, the cache then gives up the slots that
received least.

The cache is that of perf/operators.py: codes of 8 bits (e4m3, or int8) in pages [pages, kv_heads, page_size, head_dim]
and one scale for each page and head: a block's values are code * scale.  A block that is written anew takes the least
power of two with amax <= qmax * scale (qmax: 448 for e4m3, 127 for int8), at least 2^-100.
"""
import math

import numpy
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
        # one short prompt: the latency of a single user's first pass
        dict(name="prompt_one", op="prompt", B=1, T=37, pad=0, Hq=32, Hk=8, D=128, dtype="bf16", ragged=False),
        # a batch of requests of very different lengths, with unused rows behind the last one
        dict(name="prompt_packed", op="prompt", B=48, T=8190, pad=66, Hq=32, Hk=8, D=128, dtype="bf16", ragged=True),
        # small heads, a head's queries by themselves, 16-bit floats
        dict(name="prompt_small_heads", op="prompt", B=5, T=10007, pad=0, Hq=16, Hk=16, D=64, dtype="f16", ragged=True),
        # one long prompt
        dict(name="prompt_long", op="prompt", B=1, T=16384, pad=0, Hq=32, Hk=8, D=128, dtype="bf16", ragged=False),
        # a step over 64 sequences whose tokens stand at positions of three axes
        dict(name="axes_step", op="axes", B=64, N=6, Hq=32, Hk=8, D=128, dtype="bf16", rot=128, axes=3, mixed=False, pairs=False,
             norm=True, theta=1e6),
        # a prompt of text and images, the axes' frequencies interleaved
        dict(name="axes_prompt", op="axes", B=4, N=4095, Hq=32, Hk=8, D=128, dtype="bf16", rot=128, axes=3, mixed=True, pairs=False,
             norm=True, theta=5e5),
        # a decoding step over long contexts adds its tokens' attention to the sums
        dict(name="weights_step", op="weights", B=64, N=1, Hq=32, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=16384, ragged=True),
        # the last 32 tokens of 8 long prompts weigh their contexts
        dict(name="weights_window", op="weights", B=8, N=32, Hq=32, Hk=8, D=128, page=64, dtype="bf16", kind=E4M3, L=32768, ragged=True),
        # one sequence comes back to its budget
        dict(name="evict_one", op="evict", B=1, Hk=8, D=128, page=64, kind=I8, L=1100, keep=1024, first=4, last=256, ragged=False),
        # eight long prompts go into an eighth of their slots
        dict(name="evict_prompts", op="evict", B=8, Hk=8, D=128, page=64, kind=E4M3, L=32768, keep=4096, first=4, last=512, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "axes", "weights", "weights", "evict", "evict"])
    Hk, G = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8])
    D, page, kind = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), rng.choice([E4M3, I8])
    if op == "prompt":
        T = _log(rng, 1, 16384)
        c = dict(op=op, B=_log(rng, 1, min(T, 256)), T=T, pad=rng.choice([0, 0, 1, 66]), Hq=Hk * G, Hk=Hk, D=D,
                 dtype=rng.choice(["bf16", "bf16", "f16"]), ragged=rng.random() < 0.7)
        while work(c)["flops"] > 2.1e12:
            c["T"] = c["T"] * 3 // 4
        return c
    if op == "axes":
        N = _log(rng, 1, 4095)
        D = rng.choice([64, 80, 128, 128, 256])
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 16380 // N))), N=N, Hq=Hk * (G if D <= 128 and Hk * G <= 32 else 2), Hk=Hk, D=D,
                    dtype=rng.choice(["bf16", "f16", "f32"]), rot=rng.choice([D, D // 2, D // 4 * 2]), axes=rng.choice([1, 2, 3, 4]),
                    mixed=rng.random() < 0.5, pairs=rng.random() < 0.4, norm=rng.random() < 0.8, theta=rng.choice([1e4, 5e5, 1e6]))
    L = _log(rng, 1, 32768)
    if op == "weights":
        N = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 512)])
        most = min(256, int(64 * 16384 * 8 // ((L + N) * Hk)), int(3e8 // (N * Hk * G * (L + N))) + 1)
        return dict(op=op, B=_log(rng, 1, max(1, most)), N=N, Hq=Hk * G, Hk=Hk, D=D, page=page, dtype=rng.choice(["bf16", "bf16", "f16"]),
                    kind=kind, L=L, ragged=rng.random() < 0.7)
    keep = _log(rng, 1, L)
    first = rng.randint(0, min(4, keep))
    return dict(op=op, B=_log(rng, 1, max(1, min(256, 8 * 32768 // L))), Hk=Hk, D=D, page=page, kind=kind, L=L, keep=keep, first=first,
                last=rng.choice([0, (keep - first) // 2, keep - first]), ragged=rng.random() < 0.7)


def lengths(c):
    """The tokens of a packed batch's sequences: equal, or from one to thirty-two parts each; T together."""
    part = [32 ** (b / max(1, c["B"] - 1)) if c["ragged"] else 1.0 for b in range(c["B"])]
    n = [max(1, int(c["T"] * x / sum(part))) for x in part]
    n[-1] += c["T"] - sum(n)
    return [max(0, x) for x in n]


def work(case):
    c = case
    if c["op"] == "prompt":
        n = lengths(c)
        return {"bytes": sum(n) * (2 * (c["Hq"] + c["Hk"]) * c["D"] * SIZE[c["dtype"]] + 4 * c["Hq"]),
                "flops": 4 * c["D"] * c["Hq"] * sum(x * (x + 1) // 2 for x in n)}
    if c["op"] == "axes":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 4 * c["B"] * c["N"] * c["axes"], "flops": 8 * n}
    L = c["L"] * (0.75 if c["ragged"] else 1.0)
    if c["op"] == "weights":
        tokens = int(c["B"] * (L + c["N"]))
        return {"bytes": tokens * c["Hk"] * (c["D"] + 8) + c["B"] * c["N"] * c["Hq"] * (c["D"] * SIZE[c["dtype"]] + 4),
                "flops": 2 * c["N"] * c["Hq"] * c["D"] * tokens}
    rows = int(c["B"] * min(L, c["keep"]) * c["Hk"])
    return {"bytes": int(4 * c["B"] * L * c["Hk"]) + rows * (4 * c["D"] + 8), "flops": 4 * rows * c["D"]}


# ----------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _whole(g, lo, hi, shape):
    """Whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _two_to(power):
    """2^power in 32 bits by its bits, for powers from -126 to 127."""
    return (power.to(torch.int32) + 127 << 23).view(torch.float32)


def _cache(g, c, slots):
    """A pool whose pages the sequences hold in a mixed order, with codes and scales as the write gives them for normal values
    whose size differs between heads and, by a factor of two, between blocks."""
    per = -(-slots // c["page"])
    pages = c["B"] * per
    s = {"table": torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(c["B"], per)}
    shape = (pages, c["Hk"], c["page"], c["D"])
    for name in ("k", "v"):
        codes = torch.empty(shape, dtype=CODE[c["kind"]], device="cuda")
        for at in range(0, pages, 4096):
            part = torch.randn((min(4096, pages - at),) + shape[1:], generator=g, device="cuda")
            part = part.mul_(QMAX[c["kind"]] / 5).clamp_(-QMAX[c["kind"]], QMAX[c["kind"]])
            codes[at:at + 4096] = part.round_() if c["kind"] == I8 else part
        power = _whole(g, 0, 1, (pages, c["Hk"])) + _whole(g, -1, 0, (1, c["Hk"])) + round(math.log2(5 / QMAX[c["kind"]]))
        s[name], s[name + "_scale"] = codes, _two_to(power)
    return s


def _lengths(g, c, most):
    return _whole(g, -(-most // 2), most, (c["B"],)) if c["ragged"] else torch.full((c["B"],), most, dtype=torch.int32, device="cuda")


def _grid(g, c):
    """[B, N, axes]: runs of text, whose tokens stand at one position on every axis, and pictures, whose first axis stands still
    (or counts frames) while the others run over rows and columns; what follows stands behind the largest position so far."""
    B, N, A = c["B"], c["N"], c["axes"]
    wide = int(_whole(g, 3, 40, ()).item())
    text = int(_whole(g, 1, 200, ()).item())
    size = min(max(1, N // 3), wide * wide * 2)  # tokens of a picture
    unit, top = text + size, text + max(wide, -(-size // wide)) + 1
    n = torch.arange(N, device="cuda")
    run, at = n // unit, n % unit
    cell = (at - text).clamp(min=0)
    axes = [cell // (wide * wide), cell // wide % wide, cell % wide, cell % 2][:A] if A > 1 else [cell]
    pos = torch.stack([torch.where(at < text, at, text + x) for x in axes], -1) + (run * top)[:, None]
    return (pos[None] + _whole(g, 0, 5000, (B, 1, 1))).to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}
    if c["op"] == "prompt":
        # queries, keys and values as one projection gives them, side by side
        n = lengths(c)
        both = torch.randn((sum(n) + c["pad"], c["Hq"] + 2 * c["Hk"], c["D"]), generator=g, device="cuda")
        both[:, :c["Hq"]].mul_(2)
        both = both.to(DTYPE[c["dtype"]])
        s["q"], s["k"], s["v"] = both[:, :c["Hq"]], both[:, c["Hq"]:c["Hq"] + c["Hk"]], both[:, c["Hq"] + c["Hk"]:]
        order = torch.randperm(c["B"], generator=g, device="cuda").tolist()
        starts = [0]
        for b in order:
            starts.append(starts[-1] + n[b])
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        return s
    if c["op"] == "axes":
        t = DTYPE[c["dtype"]]
        s["q"] = torch.randn((c["B"], c["N"], c["Hq"], c["D"]), generator=g, device="cuda").mul_(2).to(t)
        s["k"] = torch.randn((c["B"], c["N"], c["Hk"], c["D"]), generator=g, device="cuda").mul_(2).to(t)
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(c["D"], generator=g, device="cuda")).to(t) if c["norm"] else None
        s["base"] = _whole(g, 0, 130000, (c["B"],))
        s["positions"] = _grid(g, c)
        half, A = c["rot"] // 2, c["axes"]
        i = torch.arange(half)
        s["inv_freq"] = c["theta"] ** (-i.double() / max(1, half))
        # the frequencies of an axis every few ones, or in a row (the first axis has the fewest)
        s["axis"] = (i % A if c["mixed"] else (i * (2 * A - 1) // max(1, 2 * half) + (i * 8 >= half).long()).clamp(max=A - 1)).to(torch.int32)
        return s
    L = c["L"]
    s |= _cache(g, c, L + c.get("N", 0))
    s["ctx"] = _lengths(g, c, L)
    if c["op"] == "weights":
        s["q"] = torch.randn((c["B"], c["N"], c["Hq"], c["D"]), generator=g, device="cuda").mul_(1.5).to(DTYPE[c["dtype"]])
        s["lse"] = torch.empty((c["B"], c["N"], c["Hq"]), device="cuda")
        for b, ctx in enumerate(s["ctx"].tolist()):  # as the attention over the cache leaves it
            s["lse"][b] = torch.logsumexp(_scores(s, b, ctx), -1).permute(2, 0, 1).reshape(c["N"], c["Hq"])
        s["weights"] = torch.rand((c["B"], c["Hk"], s["table"].shape[1] * c["page"]), generator=g, device="cuda")
        return s
    # sums of weights: most slots received little, some much, and some nothing at all
    shape = (c["B"], c["Hk"], s["table"].shape[1] * c["page"])
    w = torch.randn(shape, generator=g, device="cuda").mul_(2).sub_(6).exp_()
    s["weights"] = w.masked_fill_(torch.rand(shape, generator=g, device="cuda") < 0.05, 0)
    return s


# ------------------------------------------------------------------- runs
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import sampling_row_online_gb300 as lib
        if op == "prompt":
            return lib.spec_prompt_attention(s["q"], s["k"], s["v"], s["starts"], want_lse=True)
        if op == "axes":
            return lib.spec_qk_norm_rope_axes(s["q"], s["k"], s["inv_freq"], s["axis"], s["positions"], base=s["base"], norm=c["norm"],
                                              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6, pairs=c["pairs"])
        cache = lib.SpecCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "weights":
            lib.spec_cache_weights(s["q"], cache, s["table"], s["ctx"], s["lse"], s["weights"])
            return s["weights"]
        index, ctx = lib.spec_cache_evict(cache, s["table"], s["ctx"], s["weights"], c["keep"], first=c["first"], last=c["last"])
        return index, ctx, s["weights"], s["k"], s["v"], s["k_scale"], s["v_scale"]
    return {"prompt": _prompt, "axes": _axes, "weights": _weights, "evict": _evict}[op](s)


def _prompt(s):
    c = s["case"]
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    G = Hq // Hk
    out = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.full((len(out), Hq), -math.inf, device="cuda")
    starts = s["starts"].tolist()
    for lo, hi in zip(starts, starts[1:]):
        L = hi - lo
        heads = max(1, min(Hk, int(1e9 // (G * L * L + 1))))  # kv heads at a time
        later = torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1)
        for h in range(0, Hk, heads):
            k, v = (x[lo:hi, h:h + heads].float().transpose(0, 1) for x in (s["k"], s["v"]))
            q = s["q"][lo:hi, h * G:(h + heads) * G].float().reshape(L, -1, G, D).permute(1, 2, 0, 3)
            score = (q @ k[:, None].transpose(2, 3)).mul_(D ** -0.5).masked_fill_(later, -math.inf)
            top = score.amax(-1, keepdim=True)
            weight = score.sub_(top).exp_()
            total = weight.sum(-1, keepdim=True)
            x = (weight @ v[:, None]) / total
            out[lo:hi, h * G:(h + heads) * G] = x.permute(2, 0, 1, 3).reshape(L, -1, D).to(out.dtype)
            lse[lo:hi, h * G:(h + heads) * G] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(L, -1)
    return out, lse


def _axes(s):
    c = s["case"]
    r = c["rot"]
    where = (s["base"][:, None, None] + s["positions"])[..., s["axis"].long().to("cuda")]
    angle = where.double() * s["inv_freq"].to("cuda")
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, weight):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        out = y.clone()
        a, b = (slice(0, r, 2), slice(1, r, 2)) if c["pairs"] else (slice(0, r // 2), slice(r // 2, r))
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
        return out.to(x.dtype)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


def _scores(s, b, ctx):
    """[Hk, G, N, ctx + N]: the scores of sequence b's new tokens, -inf where a token does not see a slot."""
    c = s["case"]
    N, Hk, D = c["N"], c["Hk"], c["D"]
    slots = ctx + N
    pages = s["table"][b, :-(-slots // c["page"])].long()
    k = (s["k"].view(torch.uint8)[pages].view(CODE[c["kind"]]).float() * s["k_scale"][pages][..., None, None]).transpose(0, 1)
    k = k.reshape(Hk, 1, -1, D)[:, :, :slots]
    q = s["q"][b].float().reshape(N, Hk, -1, D).permute(1, 2, 0, 3)
    later = torch.arange(slots, device="cuda") > ctx + torch.arange(N, device="cuda")[:, None]
    return (q @ k.transpose(2, 3)).mul_(D ** -0.5).masked_fill_(later, -math.inf)


def _weights(s):
    c = s["case"]
    for b, ctx in enumerate(s["ctx"].tolist()):
        lse = s["lse"][b].reshape(c["N"], c["Hk"], -1).permute(1, 2, 0)[..., None]
        got = _scores(s, b, ctx).sub_(lse).exp_().sum((1, 2))
        at = s["weights"][b, :, :ctx + c["N"]]
        at[:, ctx:] = 0  # the new tokens' own slots start anew
        at += got
    return s["weights"]


def _scale_for(amax, kind):
    """The least power of two with amax <= qmax * scale, at least 2^-100."""
    half, power = torch.frexp(amax)
    top, up = math.frexp(QMAX[kind])
    power = torch.where(amax > 0, power - up + (half > top).to(power.dtype), -100)
    return _two_to(power.clamp(min=-100))


def _evict(s):
    c = s["case"]
    B, Hk, D, page, keep, kind = c["B"], c["Hk"], c["D"], c["page"], c["keep"], c["kind"]
    index = torch.full((B, Hk, keep), -1, dtype=torch.int32, device="cuda")
    left = s["ctx"].clone()
    heads = torch.arange(Hk, device="cuda")[:, None]
    for b, ctx in enumerate(s["ctx"].tolist()):
        if ctx <= keep:
            index[b, :, :ctx] = torch.arange(ctx, device="cuda")
            continue
        free = s["weights"][b, :, c["first"]:ctx - c["last"]]
        best = torch.sort(free, dim=-1, descending=True, stable=True).indices[:, :keep - c["first"] - c["last"]] + c["first"]
        ends = [torch.arange(lo, hi, device="cuda").expand(Hk, -1) for lo, hi in ((0, c["first"]), (ctx - c["last"], ctx))]
        kept = torch.cat([ends[0], best.sort(-1).values, ends[1]], 1)
        index[b] = kept
        left[b] = keep
        s["weights"][b, :, :keep] = s["weights"][b].gather(1, kept)
        blocks = -(-keep // page)
        source, row, to = s["table"][b].long()[kept // page], kept % page, s["table"][b, :blocks].long()
        for name in ("k", "v"):
            codes, scales = s[name].view(torch.uint8), s[name + "_scale"]
            x = codes[source, heads, row].view(CODE[kind]).float() * scales[source, heads][..., None]
            full = torch.zeros((Hk, blocks * page, D), device="cuda")
            full[:, :keep] = x
            scale = _scale_for(full.reshape(Hk, blocks, -1).abs().amax(-1), kind)
            x = x / scale.repeat_interleave(page, 1)[:, :keep, None]
            x = x.round().clamp(-127, 127).to(torch.int8) if kind == I8 else x.to(torch.float8_e4m3fn)
            slot = torch.arange(keep, device="cuda")
            codes[to[slot // page][None], heads, (slot % page)[None]] = x.view(torch.uint8)
            scales[to] = scale.T
    return index, left, s["weights"], s["k"], s["v"], s["k_scale"], s["v_scale"]


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """In 64 bits, from the definitions."""
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "axes": _exact_axes, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _exact_prompt(s):
    c = s["case"]
    if work(c)["flops"] > 6e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for b in range(c["B"]):
        for i in range(starts[b], starts[b + 1], 512):  # 512 tokens at a time see what stands up to the last of them
            j = min(i + 512, starts[b + 1])
            k, v = (x[starts[b]:j].double() for x in (s["k"], s["v"]))
            hidden = torch.arange(starts[b], j, device="cuda")[None, :] > torch.arange(i, j, device="cuda")[:, None]
            for h in range(c["Hq"]):
                kv = h * c["Hk"] // c["Hq"]
                x = torch.where(hidden, -math.inf, s["q"][i:j, h].double() @ k[:, kv].T / math.sqrt(c["D"]))
                lse[i:j, h] = x.logsumexp(1)
                out[i:j, h] = x.softmax(1) @ v[:, kv]
    return out, lse


def _exact_axes(s):
    c = s["case"]
    r = c["rot"]
    where = s["base"].double()[:, None, None] + s["positions"].double()
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if c["norm"]:
            y = y / (y.square().sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + r // 2)
            angle = (where[..., int(s["axis"][i])] * float(s["inv_freq"][i]))[..., None]
            y[..., a], y[..., b] = y[..., a] * angle.cos() - y[..., b] * angle.sin(), y[..., b] * angle.cos() + y[..., a] * angle.sin()
        got.append(y)
    return tuple(got)


def _exact_row(s, name, b, h, slots):
    """[slots, D] in 64 bits: the values that sequence b's head h holds in `slots` (numbers)."""
    c = s["case"]
    slots = torch.as_tensor(slots, device="cuda")
    page = s["table"][b][slots // c["page"]].long()
    return s[name].view(torch.uint8)[page, h, slots % c["page"]].view(CODE[c["kind"]]).double() * s[name + "_scale"][page, h].double()[:, None]


def _exact_weights(s):
    c = s["case"]
    if work(c)["flops"] > 6e11 or c["B"] * c["Hk"] * c["N"] > 20000:
        return None
    G = c["Hq"] // c["Hk"]
    got = s["weights"].double()
    for b, ctx in enumerate(s["ctx"].tolist()):
        for h in range(c["Hk"]):
            keys = _exact_row(s, "k", b, h, range(ctx + c["N"]))
            got[b, h, ctx:ctx + c["N"]] = 0
            for i in range(c["N"]):
                x = s["q"][b, i, h * G:(h + 1) * G].double() @ keys[:ctx + i + 1].T / math.sqrt(c["D"])
                got[b, h, :ctx + i + 1] += (x - s["lse"][b, i, h * G:(h + 1) * G].double()[:, None]).exp().sum(0)
    return got


def _exact_rounding(x, kind):
    """x (64 bits, within the codes' range) to the nearest code value, ties to even: the spacing is 1, or that of e4m3 at x."""
    if kind == I8:
        return torch.round(x)
    at = torch.tensor([2.0 ** e for e in range(-6, 9)], dtype=torch.float64, device="cuda")
    step = at[torch.searchsorted(at, x.abs(), right=True).clamp(min=1) - 1] / 8
    return torch.round(x / step) * step


def _exact_evict(s):
    c = s["case"]
    if s["k"].numel() > 8e8 or c["B"] * c["Hk"] * (c["keep"] // c["page"] + 8) > 20000:
        return None
    held = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale", "weights")}
    scales = torch.tensor([2.0 ** e for e in range(-100, 128)], dtype=torch.float64, device="cuda")
    weights, table = s["weights"].cpu().numpy(), s["table"].tolist()
    for b, ctx in enumerate(s["ctx"].tolist()):
        if ctx <= c["keep"]:
            continue
        for h in range(c["Hk"]):
            slot = numpy.arange(ctx)
            given = (slot < c["first"]) | (slot >= ctx - c["last"])
            order = numpy.lexsort((slot, -weights[b, h, :ctx].astype(numpy.float64), ~given))
            kept = numpy.sort(order[:c["keep"]])
            held["weights"][b, h, :c["keep"]] = torch.from_numpy(weights[b, h][kept]).double().cuda()
            for name in ("k", "v"):
                rows = _exact_row(s, name, b, h, kept)
                for at in range(0, c["keep"], c["page"]):
                    part = rows[at:at + c["page"]]
                    scale = scales[torch.searchsorted(scales * QMAX[c["kind"]], part.abs().amax())]
                    held[name + "_scale"][table[b][at // c["page"]], h] = scale
                    held[name][table[b][at // c["page"]], h, :len(part)] = _exact_rounding(part / scale, c["kind"])
    whole = c["kind"] == I8  # whole numbers have no 64-bit value to be compared with
    return (None, None, held["weights"]) + tuple(None if whole and n in ("k", "v") else held[n] for n in ("k", "v", "k_scale", "v_scale"))
