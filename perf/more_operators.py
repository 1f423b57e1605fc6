"""Workloads of the attention side of a layer, with their plain forms: rotary
positions, a paged key/value cache in 4 bits (written and read back), and
attention over that cache.

Rotary positions.  Pair i of a head turns by the angle p f_i at position p:
y1 = m (x1 cos - x2 sin), y2 = m (x1 sin + x2 cos).  The pairs are the first
`part` elements of a head, i with i + part / 2 ("half") or 2 i with 2 i + 1
("interleaved"); the rest of the head stays.  A program holds the frequencies as
turns per position in 64-bit fixed point, round(f / (2 pi) 2^64).

The cache.  A token has one row of k and one of v for each key/value head, in a
4-bit format:

  mxfp4   E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), blocks of 32
          with scale 2^(byte - 127), byte = floor(log2 max|x|) - 2 + 127; the
          row's exponent is its largest byte - 127
  nvfp4   the same codes, blocks of 16 with scale E4M3 = max|x| / (6 2^e) to
          nearest, e for each row: the least with max|row| <= 2688 2^e

Values round to the nearest code, ties to the even one, and saturate at 6.  Rows
are stored with the head dimension filled up to 64, 128 or 256, in pages of
page_size tokens: codes (pages, 2, heads, page_size, width / 2) with the even
element in the low nibble, scales (pages, 2, heads, page_size, width / block),
exponents (int8) (pages, 2, heads, page_size); 0 is k and 1 is v.

A batch.  Sequence b has lengths[b] tokens in the cache, the pages page_table[b],
and the new tokens starts[b] .. starts[b + 1] of the call, which are its last.

Attention.  A query at position p sees the tokens j <= p of its sequence; with a
window w those with j > p - w or j < sinks.
"""
import math

import torch

own = False

FORMATS = {"mxfp4": 32, "nvfp4": 16}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- the cases -------------------------------------------------------------

def listed():
    return [
        # the queries and keys of one new token, far into a conversation
        {"name": "rotary, one token", "kind": "rotary", "tokens": 1, "heads": 40, "more": 8, "dim": 128, "part": 128, "interleaved": False, "type": "bf16",
         "base": 10000.0, "scaling": "none", "factor": 1.0, "far": 100000, "train": False},
        # a layer of a large model in training: its queries and keys, there and back
        {"name": "rotary, training", "kind": "rotary", "tokens": 8192, "heads": 40, "more": 8, "dim": 128, "part": 128, "interleaved": True, "type": "bf16",
         "base": 500000.0, "scaling": "none", "factor": 1.0, "far": 8192, "train": True},
        # fine tuning for a longer context, a quarter of an odd head
        {"name": "rotary, ragged", "kind": "rotary", "tokens": 1009, "heads": 25, "more": 0, "dim": 80, "part": 20, "interleaved": False, "type": "f32",
         "base": 10000.0, "scaling": "bands", "factor": 8.0, "far": 65536, "train": True},
        # a server's step: one new token for each of its requests, with rotated keys
        {"name": "cache, one token each", "kind": "cache", "fmt": "nvfp4", "batch": 32, "most": 1, "least": 1, "longest": 8192, "shortest": 16, "heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "rotary": True, "interleaved": False},
        # a long prompt
        {"name": "cache, a prompt", "kind": "cache", "fmt": "mxfp4", "batch": 1, "most": 8192, "least": 8192, "longest": 8192, "shortest": 8192, "heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "rotary": True, "interleaved": False},
        # further turns of some conversations, heads of 96
        {"name": "cache, ragged", "kind": "cache", "fmt": "nvfp4", "batch": 5, "most": 333, "least": 1, "longest": 4099, "shortest": 17, "heads": 3, "dim": 96,
         "page": 16, "type": "f16", "rotary": False, "interleaved": False},
        # the first tokens of a single short answer: latency
        {"name": "attend, one short", "kind": "attend", "fmt": "mxfp4", "batch": 1, "most": 1, "least": 1, "longest": 523, "shortest": 523, "heads": 8, "group": 4, "dim": 128,
         "page": 16, "type": "bf16", "window": 0, "sinks": 0},
        # a server's step over requests of very different lengths
        {"name": "attend, a batch", "kind": "attend", "fmt": "mxfp4", "batch": 64, "most": 1, "least": 1, "longest": 8192, "shortest": 100, "heads": 8, "group": 8, "dim": 128,
         "page": 64, "type": "bf16", "window": 0, "sinks": 0},
        # one long document
        {"name": "attend, one long", "kind": "attend", "fmt": "nvfp4", "batch": 1, "most": 1, "least": 1, "longest": 131071, "shortest": 131071, "heads": 8, "group": 8, "dim": 128,
         "page": 256, "type": "bf16", "window": 0, "sinks": 0},
        # a step of a model with local layers, a few proposed tokens each
        {"name": "attend, a window", "kind": "attend", "fmt": "nvfp4", "batch": 32, "most": 4, "least": 1, "longest": 32768, "shortest": 1000, "heads": 4, "group": 4, "dim": 64,
         "page": 32, "type": "f16", "window": 1000, "sinks": 4},
        # a long prompt
        {"name": "attend, a prompt", "kind": "attend", "fmt": "mxfp4", "batch": 1, "most": 8192, "least": 8192, "longest": 8192, "shortest": 8192, "heads": 8, "group": 4, "dim": 128,
         "page": 64, "type": "bf16", "window": 0, "sinks": 0},
        # further parts of long prompts, wide heads
        {"name": "attend, chunks", "kind": "attend", "fmt": "nvfp4", "batch": 3, "most": 700, "least": 100, "longest": 16000, "shortest": 2111, "heads": 2, "group": 5, "dim": 256,
         "page": 64, "type": "f16", "window": 0, "sinks": 0},
    ]


def draw(rng):
    def size(low, high):
        """Spread over the logarithm; a multiple of 64 or of 8 half of the time, any number otherwise."""
        x = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        to = rng.choice((64, 8, 1, 1))
        return min(high, max(low, -(-x // to) * to))

    kind = rng.choice(("rotary", "rotary", "cache", "cache", "attend", "attend", "attend", "attend"))
    dim = rng.choice((64, 96, 128, 128, 128, 256))
    if kind == "rotary":
        dim = rng.choice((dim, 80))
        part = rng.choice((dim, dim, dim // 2, dim // 4))
        scaling = rng.choice(("none", "linear", "base", "bands"))
        return {"kind": kind, "tokens": size(1, 8192), "heads": rng.randint(1, 40), "more": rng.choice((0, 8)), "dim": dim, "part": part, "interleaved": rng.random() < 0.5,
                "type": rng.choice(("bf16", "bf16", "f16", "f32")), "base": rng.choice((10000.0, 500000.0)), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice((2.0, 8.0, 32.0)), "far": size(100, 1 << 20), "train": rng.random() < 0.5}
    case = {"kind": kind, "fmt": rng.choice(("mxfp4", "nvfp4")), "heads": rng.choice((1, 2, 3, 8, 8)), "dim": dim, "page": rng.choice((16, 32, 64, 256)),
            "type": rng.choice(("bf16", "bf16", "f16"))}
    if kind == "cache":
        batch = size(1, 64)
        most = size(1, 8192 // batch)
        longest = most + size(1, 8192)
        case.update(batch=batch, most=most, least=rng.randint(1, most), longest=longest, shortest=rng.randint(most, longest), rotary=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5)
        if rng.random() < 0.3:
            case["type"] = "f32"
        return case
    case["group"] = rng.choice((1, 2, 4, 5, 8, 8, 16))
    case["window"], case["sinks"] = rng.choice(((0, 0), (0, 0), (size(16, 4096), rng.choice((0, 1, 4, 20)))))
    if rng.random() < 0.65:  # a step: one new token or a few
        batch, most = size(1, 64), rng.choice((1, 1, 2, 5))
        longest = size(16, min(131072, (64 * 4096 * 8 * 128) // (batch * case["heads"] * dim)))
    else:  # prompts or parts of them
        batch = size(1, 8)
        most = size(16, 4096 // batch)
        longest = most + rng.choice((0, size(1, 4096)))
    case.update(batch=batch, most=most, least=rng.randint(1, most), longest=longest, shortest=rng.randint(1, longest))
    return case


def spread(most, least, count, step):
    """`count` sizes from `most` down to `least`, in no order."""
    return [most - int((most - least) * (i * step % 1.0)) for i in range(count)]


def batch_of(case):
    """(length, new tokens) of each sequence."""
    lengths = spread(case["longest"], case["shortest"], case["batch"], 0.6180339887)
    return [(n, min(n, m)) for n, m in zip(lengths, spread(case["most"], case["least"], case["batch"], 0.7548776662))]


def width_of(dim):
    return 64 if dim <= 64 else 128 if dim <= 128 else 256


def seen(case, p):
    """How many tokens a query at position p sees."""
    w = case["window"]
    if w == 0 or p < w:
        return p + 1
    return w + min(case["sinks"], p + 1 - w)


def work(case):
    kind, size = case["kind"], TYPES[case["type"]].itemsize
    if kind == "rotary":
        n = case["tokens"] * case["heads"] * case["dim"] * (2 if case["train"] else 1)
        return {"bytes": 2 * n * size, "flops": 3.0 * n * case["part"] / case["dim"]}
    stored = case["dim"] * (0.5 + 1 / FORMATS[case["fmt"]]) + 1  # bytes of a row
    batch = batch_of(case)
    if kind == "cache":
        rows = 2 * case["heads"] * sum(n for _, n in batch)
        # values in, rows out, and the values they stand for (bf16)
        return {"bytes": rows * (case["dim"] * (size + 2) + 2 * stored), "flops": 0}
    heads = case["heads"] * case["group"]
    need = pairs = 0
    for length, n in batch:
        p = length - n
        need += seen(case, p) + n - 1
        if case["window"] == 0:
            pairs += n * (p + 1) + n * (n - 1) // 2
        else:
            pairs += sum(seen(case, i) for i in range(p, length))
    rows = heads * sum(n for _, n in batch)
    return {"bytes": 2 * case["heads"] * need * stored + 2 * rows * case["dim"] * size, "flops": 4.0 * pairs * heads * case["dim"]}


# ---- inputs ----------------------------------------------------------------

def frequencies(case):
    """The turning rates of the pairs, in radians per position (64 bits)."""
    part, base, factor = case["part"], case["base"], case["factor"]
    if case["scaling"] == "base":
        base *= factor ** (part / (part - 2))
    f = base ** (-torch.arange(0, part, 2, dtype=torch.float64) / part)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "bands":  # pairs of 32 turns and more over the 4096 positions of before stay, of one and fewer are stretched
        keep = ((f * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f


def magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "bands" else 1.0


def turning(f, m, interleaved):
    """The plan of a rotation: frequencies, and the same in 64-bit fixed point."""
    return {"f": f.cuda(), "turns": (f / (2 * math.pi) * 2.0 ** 64).to(torch.int64).cuda(), "m": m, "interleaved": interleaved}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    kind, dim = case["kind"], case["dim"]
    if kind == "rotary":
        t, h = case["tokens"], case["heads"]
        # the queries and keys are a part of what one product gave; so may be the gradients
        fused = normal(2, t, h + case["more"], dim).to(dtype)
        s = dict(case, x=fused[0, :, :h], plan=turning(frequencies(case), magnitude(case), case["interleaved"]))
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
        if case["train"]:
            s["dy"] = fused[1, :, :h].contiguous()
        return s

    batch, page, heads = batch_of(case), case["page"], case["heads"]
    starts = [0]
    for _, n in batch:
        starts.append(starts[-1] + n)
    need = [-(-length // page) for length, _ in batch]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(batch), max(need)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):][:n]
    s = dict(case, tokens=starts[-1], most_new=max(n for _, n in batch), most_seen=max(n for n, _ in batch), table=table)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lengths"] = torch.tensor([n for n, _ in batch], dtype=torch.int32, device="cuda")
    channels = torch.exp(0.5 * normal(2, heads, 1, dim))  # of unequal size, as keys and values have them
    width = width_of(dim)
    if kind == "cache":
        values = normal(2, starts[-1], heads, dim) * channels.view(2, 1, heads, dim)
        s["k"], s["v"] = (x.contiguous() for x in values.to(dtype))
        rows = torch.zeros(pages, 2, heads, page, width, device="cuda")
        if case["rotary"]:
            s["plan"] = turning(frequencies(dict(part=dim, base=500000.0, factor=1.0, scaling="none")), 1.0, case["interleaved"])
    else:
        rows = torch.nn.functional.pad(normal(pages, 2, heads, page, dim) * channels, (0, width - dim))
        s["q"] = normal(starts[-1], heads * case["group"], dim).to(dtype)
    s["cache"] = stored(rows, case["fmt"], dim)
    return s


def scaled_blocks(x, fmt):
    """Rows x (..., k), k whole blocks, in 32 bits as (codes' values, scales, row exponents): (..., blocks, size), (..., blocks), (...)."""
    size = FORMATS[fmt]
    x = x.float().unflatten(-1, (-1, size))
    most = x.abs().amax(-1)
    if fmt == "mxfp4":
        e = torch.zeros(most.shape[:-1], dtype=torch.int32, device=x.device)
        scale = torch.exp2(torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127).float())
        y = x / torch.where(scale > 0, scale, 1.0)[..., None]
    else:
        top = most.amax(-1)
        m, ex = torch.frexp(top)
        e = torch.where(top > 0, torch.where(m <= 0.65625, ex - 12, ex - 11), 0).clamp(min=-100).to(torch.int32)
        unit = torch.exp2(-e.float())[..., None]
        a = most * unit / 6
        step = torch.exp2((torch.frexp(a).exponent - 4).clamp(min=-9).float())
        scale = torch.where(most > 0, (torch.round(a / step) * step).clamp(2.0 ** -9, 448.0), 0.0)
        y = x * unit[..., None] / torch.where(scale > 0, scale, 1.0)[..., None]
    y = y.clamp(-6.0, 6.0)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return torch.round(y / step) * step, scale, e


def stored(x, fmt, dim):
    """Rows (pages, 2, heads, page_size, width) as a program's cache holds them."""
    y, scale, e = scaled_blocks(x, fmt)
    a = y.abs()
    code = (torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (y < 0).to(torch.uint8) << 3).flatten(-2)
    m, ex = torch.frexp(scale)
    if fmt == "mxfp4":
        byte = torch.where(scale > 0, ex + 126, 0)
        e = byte.amax(-1) - 127
    else:  # E4M3: subnormals count in steps of 2^-9
        byte = torch.where(scale < 2.0 ** -6, scale * 512, (ex + 6) * 8 + (m * 16 - 8))
    return {"codes": (code[..., 0::2] | code[..., 1::2] << 4).contiguous(), "scales": byte.to(torch.uint8), "exponents": e.to(torch.int8),
            "head_dim": dim, "fmt": fmt}


def stood_for(codes, scales, exponents, fmt, dtype=torch.float32):
    """The values of stored rows (..., width)."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device, dtype=dtype)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()].unflatten(-1, (-1, FORMATS[fmt]))
    byte = scales.to(dtype)
    if fmt == "mxfp4":
        return (v * torch.exp2(byte - 127)[..., None]).flatten(-2)
    m, ex = byte % 8, torch.floor(byte / 8)
    scale = torch.where(ex > 0, (8 + m) * torch.exp2(ex - 10), m * 2.0 ** -9)
    return (v * scale[..., None]).flatten(-2) * torch.exp2(exponents.to(dtype))[..., None]


# ---- one pass --------------------------------------------------------------

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import extended_precision_gemm_gb300 as ddg

    def rotation():
        p = s["plan"]
        return ddg.Rotary(p["turns"], scale=p["m"], interleaved=p["interleaved"])

    if s["kind"] == "rotary":
        y = ddg.rotary(s["x"], s["positions"], rotation())
        return {"y": y, "dx": ddg.rotary_backward(s["dy"], s["positions"], rotation())} if s["train"] else y
    cache = ddg.MX4Cache(**s["cache"])
    if s["kind"] == "cache":
        ddg.mx4_cache_append(cache, s["k"], s["v"], s["starts"], s["lengths"], s["table"], rotary=rotation() if s["rotary"] else None)
        return ddg.mx4_cache_read(cache, s["tokens"], s["starts"], s["lengths"], s["table"], dtype=torch.bfloat16)
    return ddg.mx4_attention(s["q"], cache, s["starts"], s["lengths"], s["table"], window=s["window"], sinks=s["sinks"])


def turned(x, positions, plan, back=False):
    """x (tokens, heads, dim) rotated, in x's precision; the angles in 64 bits."""
    angle = positions.double()[:, None, None] * plan["f"]
    c, s = (plan["m"] * torch.cos(angle)).to(x.dtype), (plan["m"] * torch.sin(angle)).to(x.dtype)
    s = -s if back else s
    half = plan["f"].numel()
    if plan["interleaved"]:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : 2 * half]
        y = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((y, x[..., 2 * half :]), -1)


def places(s):
    """(sequence, index among its new tokens, position) of each new token."""
    starts = s["starts"].long()
    token = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(starts, token, right=True) - 1
    i = token - starts[b]
    return b, i, s["lengths"].long()[b] - (starts[b + 1] - starts[b]) + i


def run_plain(s):
    if s["kind"] == "rotary":
        y = turned(s["x"].float(), s["positions"], s["plan"]).to(s["x"].dtype)
        return {"y": y, "dx": turned(s["dy"].float(), s["positions"], s["plan"], back=True).to(y.dtype)} if s["train"] else y
    b, i, position = places(s)
    fmt, dim = s["fmt"], s["dim"]
    cache, page = s["cache"], s["page"]
    if s["kind"] == "cache":
        k = s["k"]
        if s["rotary"]:  # values next to a border between two codes: in 64 bits
            k = turned(k.double(), position, s["plan"])
        values = torch.nn.functional.pad(torch.stack((k.float(), s["v"].float()), 1), (0, width_of(dim) - dim))
        new = stored(values, fmt, dim)
        at, off = s["table"][b, position // page].long(), position % page
        for name in ("codes", "scales", "exponents"):
            cache[name][at, :, :, off] = new[name]
        rows = [cache[name][at, :, :, off] for name in ("codes", "scales", "exponents")]
        values = stood_for(*rows, fmt)[..., :dim].to(torch.bfloat16)
        return values[:, 0].contiguous(), values[:, 1].contiguous()

    # every sequence filled up to the longest: (batch, heads, tokens, dim)
    most = s["most_seen"]
    j = torch.arange(most, device="cuda")
    at, off = s["table"][:, j // page].clamp(min=0).long(), j % page
    rows = [cache[name][at, :, :, off] for name in ("codes", "scales", "exponents")]
    k, v = stood_for(*rows, fmt)[..., :dim].permute(2, 0, 3, 1, 4)
    heads, group = s["heads"], s["group"]
    q = torch.zeros(s["batch"], s["most_new"], heads, group, dim, device="cuda")
    q[b, i] = s["q"].float().view(-1, heads, group, dim)
    p = torch.full((s["batch"], s["most_new"]), -1, dtype=torch.int64, device="cuda")
    p[b, i] = position
    sees = j <= p[..., None]
    if s["window"]:
        sees &= (j > p[..., None] - s["window"]) | (j < s["sinks"])
    score = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.mT * dim ** -0.5  # (batch, heads, new x group, tokens)
    sees = sees[:, None, :, None].expand(-1, -1, -1, group, -1).flatten(2, 3)
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    score = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = score.sum(-1, keepdim=True)
    y = score @ torch.where((j < s["lengths"][:, None])[:, None, :, None], v, 0.0) / torch.where(total > 0, total, 1.0)
    return y.unflatten(2, (-1, group)).permute(0, 2, 1, 3, 4)[b, i].flatten(1, 2).to(s["q"].dtype)


# ---- the definition in 64 bits ---------------------------------------------

def nearest(x, fmt):
    """Rows x (rows, k) in 64 bits after quantisation: each block against the list of codes."""
    rows, k = x.shape
    size = FORMATS[fmt]
    x = torch.cat((x, torch.zeros(rows, -k % size, dtype=torch.float64, device=x.device)), 1).reshape(rows, -1, size)
    most = x.abs().max(2, keepdim=True).values
    some = torch.where(most > 0, most, 1.0)
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(some))
        e = torch.where(torch.exp2(e) > some, e - 1, torch.where(torch.exp2(e + 1) <= some, e + 1, e))
        unit = torch.exp2((e - 2).clamp(-127, 127))
    else:
        top = most.max(1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 2688))
        e = torch.where(torch.exp2(e - 1) * 2688 >= top, e - 1, torch.where(torch.exp2(e) * 2688 < top, e + 1, e))
        e = torch.where(top > 0, e, 0.0).clamp(min=-100)
        grid = torch.cat([torch.arange(8, dtype=torch.float64) * 2.0 ** -9] + [(8 + torch.arange(8, dtype=torch.float64)) * 2.0 ** (p - 10) for p in range(1, 16)])[:127].to(x.device)
        want = most / 6 * torch.exp2(-e)
        up = torch.searchsorted(grid, want.contiguous()).clamp(1, 126)  # grid[up - 1] < want <= grid[up]
        low, high = want - grid[up - 1], grid[up] - want
        at = torch.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up).clamp(min=1)
        unit = grid[at] * torch.exp2(e)
    y = (x / unit).abs()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    code = torch.zeros_like(y, dtype=torch.int64)
    for i in range(7):
        code += (y >= mids[i]) if i % 2 else (y > mids[i])
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    return (table[code] * torch.sign(x) * unit).reshape(rows, -1)[:, :k]


def rotation_matrices(x, positions, f, m, interleaved, sign):
    """x (tokens, heads, dim) with each pair as a complex number times m exp(i sign p f)."""
    n = f.numel()
    angle = sign * positions.double()[:, None] * f
    turn = torch.polar(torch.full_like(angle, m), angle)[:, None]
    x = x.double()
    if interleaved:
        z = torch.view_as_complex(x[..., : 2 * n].unflatten(-1, (n, 2)).contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :n].contiguous(), x[..., n : 2 * n].contiguous()) * turn
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., 2 * n :]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rotary":
        f, m, inter = s["plan"]["f"], s["plan"]["m"], case["interleaved"]
        y = rotation_matrices(s["x"], s["positions"], f, m, inter, 1)
        return {"y": y, "dx": rotation_matrices(s["dy"], s["positions"], f, m, inter, -1)} if case["train"] else y
    batch = batch_of(case)
    if kind == "cache":
        k, v = s["k"].double(), s["v"].double()
        if case["rotary"]:
            p = torch.cat([torch.arange(length - n, length) for length, n in batch]).cuda()
            k = rotation_matrices(k, p, s["plan"]["f"], 1.0, case["interleaved"], 1)
        return tuple(nearest(x.reshape(-1, case["dim"]), case["fmt"]).reshape(x.shape) for x in (k, v))
    out, at = [], 0
    for b, (length, n) in enumerate(batch):
        used = s["table"][b, : -(-length // case["page"])].long()
        rows = [s["cache"][name][used].movedim(3, 1).flatten(0, 1)[:length] for name in ("codes", "scales", "exponents")]
        kv = stood_for(*rows, case["fmt"], torch.float64)[..., : case["dim"]]  # (length, 2, heads, dim)
        q = s["q"][at : at + n].double().unflatten(1, (case["heads"], case["group"]))
        at += n
        p = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        hidden = j > p
        if case["window"]:
            hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
        heads = []
        for h in range(case["heads"]):
            score = torch.einsum("ngd,ld->ngl", q[:, h], kv[:, 0, h]) / math.sqrt(case["dim"])
            weight = torch.softmax(score.masked_fill_(hidden[:, None], -math.inf), -1)
            heads.append(torch.einsum("ngl,ld->ngd", weight, kv[:, 1, h]))
        out.append(torch.cat(heads, 1))
    return torch.cat(out)
