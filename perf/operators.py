"""Workloads of the 4-bit microscaled products and of the gated feed-forward
block, with their plain forms.

Formats.  A matrix in 4-bit microscaled form holds E2M1 codes (0, 0.5, 1, 1.5,
2, 3, 4, 6 and their negatives), two to a byte along k (the even k in the low
nibble), and one scale for every block of k:

  mxfp4   blocks of 32, scale 2^(byte - 127), byte = floor(log2 max|x|) - 2 + 127
  nvfp4   blocks of 16, scale E4M3 = max|x| / (6 * 2^e) rounded to nearest, with
          an exponent e for each row: the least e with max|row| <= 2688 * 2^e

Values round to the nearest code, ties to the even one, and saturate at 6.
Scales are stored in tiles of 128 rows by 4 blocks (512 bytes: row r, block b
at (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4), k padded to 256 with zeros.

The gated block is y = (act(x Wg^T) * (x Wu^T)) Wd^T.  Its 4-bit form holds Wg
and Wu in one matrix, 32 rows of one and 32 of the other in turn (the last
groups filled up with zeros).
"""
import math

import torch

own = False

FORMATS = {"mxfp4": 32, "nvfp4": 16}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- the cases -------------------------------------------------------------

def listed():
    return [
        # the input of a layer for one new token
        {"name": "quantise one token", "kind": "quantise", "rows": 1, "k": 8192, "type": "bf16", "fmt": "mxfp4", "cols": False},
        # a large weight matrix, once after training
        {"name": "quantise a weight matrix", "kind": "quantise", "rows": 8192, "k": 16384, "type": "bf16", "fmt": "nvfp4", "cols": True},
        # a layer's product for one new token: the weights are read once
        {"name": "product, one token", "kind": "product", "m": 1, "n": 8192, "k": 8192, "fmt": "nvfp4", "type": "bf16"},
        # a short prompt of odd length on a width that fills no tile
        {"name": "product, ragged", "kind": "product", "m": 333, "n": 2050, "k": 4100, "fmt": "mxfp4", "type": "f16"},
        # a long prompt, or the batch of a server at full load
        {"name": "product, large", "kind": "product", "m": 8192, "n": 8192, "k": 8192, "fmt": "nvfp4", "type": "bf16"},
        # a small model's training step
        {"name": "train, small", "kind": "train", "t": 96, "d": 256, "f": 640, "type": "bf16", "act": "silu"},
        # a large model's training step
        {"name": "train, large", "kind": "train", "t": 8192, "d": 4096, "f": 12288, "type": "bf16", "act": "silu"},
        # one new token through the 16-bit block
        {"name": "forward, one token", "kind": "forward", "t": 1, "d": 4096, "f": 12288, "type": "bf16", "act": "silu"},
        # a prompt of odd length through a block of odd widths
        {"name": "forward, ragged", "kind": "forward", "t": 1009, "d": 2056, "f": 5400, "type": "f16", "act": "gelu"},
        # one new token through the 4-bit block
        {"name": "serve, one token", "kind": "serve", "t": 1, "d": 4096, "f": 12288, "type": "bf16", "act": "silu", "fmt": "mxfp4"},
        # the new tokens of a batch of requests
        {"name": "serve, a batch", "kind": "serve", "t": 45, "d": 4096, "f": 12288, "type": "bf16", "act": "silu", "fmt": "nvfp4"},
        # a prompt through the 4-bit block
        {"name": "serve, a prompt", "kind": "serve", "t": 4096, "d": 4096, "f": 12288, "type": "bf16", "act": "gelu_tanh", "fmt": "mxfp4"},
    ]


def draw(rng):
    def size(low, high):
        """Spread over the logarithm; a multiple of 64 or of 8 half of the time, any number otherwise."""
        x = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        to = rng.choice((64, 8, 1, 1))
        x = min(high, max(low, -(-x // to) * to))
        return x + 64 if x == 3072 else x

    kind = rng.choice(("quantise", "product", "product", "train", "forward", "serve"))
    if kind == "quantise":
        rows, k = size(1, 8192), size(16, 16384)
        return {"kind": kind, "rows": rows, "k": k, "type": rng.choice(("bf16", "f16", "f32")), "fmt": rng.choice(("mxfp4", "nvfp4")), "cols": rng.random() < 0.5}
    if kind == "product":
        return {"kind": kind, "m": size(1, 8192), "n": size(16, 8192), "k": size(16, 8192), "fmt": rng.choice(("mxfp4", "nvfp4")), "type": rng.choice(("bf16", "f16", "f32"))}
    act = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu"))
    t, d, f = size(1, 8192), size(64, 4096), size(128, 12288)
    case = {"kind": kind, "t": t, "d": d, "f": f, "type": rng.choice(("bf16", "bf16", "f16")), "act": act}
    if kind == "serve":
        case["fmt"] = rng.choice(("mxfp4", "nvfp4"))
    return case


def work(case):
    kind = case["kind"]
    if kind == "quantise":
        n = case["rows"] * case["k"]
        # x in, codes and scales out, and the values they stand for (bf16)
        return {"bytes": n * (TYPES[case["type"]].itemsize + 0.5 + 1 / FORMATS[case["fmt"]] + 2), "flops": 0}
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * (0.5 + 1 / FORMATS[case["fmt"]]) + m * n * TYPES[case["type"]].itemsize, "flops": 2.0 * m * n * k}
    t, d, f = case["t"], case["d"], case["f"]
    if kind == "serve":
        return {"bytes": 3 * d * f * (0.5 + 1 / FORMATS[case["fmt"]]) + 2 * 2 * t * d, "flops": 6.0 * t * d * f}
    if kind == "forward":
        return {"bytes": 2 * (3 * d * f + 2 * t * d), "flops": 6.0 * t * d * f}
    # x, dy and the weights in; y, dx and the weights' gradients out
    return {"bytes": 2 * (6 * d * f + 4 * t * d), "flops": 18.0 * t * d * f}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]

    def normal(rows, cols, scale=1.0):
        return torch.randn(rows, cols, generator=g, device="cuda") * scale

    def activations(rows, cols):
        """Channels of unequal size, as a layer's inputs have them."""
        return normal(rows, cols) * torch.exp(0.5 * normal(1, cols))

    kind = case["kind"]
    if kind == "quantise":
        shape = (case["k"], case["rows"]) if case["cols"] else (case["rows"], case["k"])
        return dict(case, x=activations(*shape).to(dtype))
    if kind == "product":
        fmt = case["fmt"]
        return dict(case, a=stored(activations(case["m"], case["k"]), fmt), b=stored(normal(case["n"], case["k"], case["k"] ** -0.5), fmt))
    t, d, f = case["t"], case["d"], case["f"]
    s = dict(case, x=activations(t, d).to(dtype))
    weights = normal(f, d, d ** -0.5), normal(f, d, d ** -0.5), normal(d, f, f ** -0.5)
    if kind == "serve":  # quantised once, when the model was loaded
        pair = [torch.nn.functional.pad(w, (0, 0, 0, -f % 32)).view(-1, 32, d) for w in weights[:2]]
        s["w_in"], s["w_out"] = stored(torch.stack(pair, 1).view(-1, d), case["fmt"]), stored(weights[2], case["fmt"])
    else:
        s["wg"], s["wu"], s["wd"] = (w.to(dtype) for w in weights)
    if kind == "train":
        s["dy"] = normal(t, d).to(dtype)
    return s


def scaled_blocks(x, fmt):
    """x (rows, k) in 32 bits as (codes' values, scales, row exponents): (rows, blocks, size), (rows, blocks), (rows,)."""
    rows, k = x.shape
    size = FORMATS[fmt]
    x = torch.nn.functional.pad(x.float(), (0, -k % size)).view(rows, -1, size)
    most = x.abs().amax(2)
    if fmt == "mxfp4":
        e = torch.zeros(rows, dtype=torch.int32, device=x.device)
        scale = torch.exp2(torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127).float())
        y = x / torch.where(scale > 0, scale, 1.0)[..., None]
    else:
        top = most.amax(1)
        m, ex = torch.frexp(top)
        e = torch.where(top > 0, torch.where(m <= 0.65625, ex - 12, ex - 11), 0).clamp(min=-100).to(torch.int32)
        unit = torch.exp2(-e.float())[:, None]
        a = most * unit / 6
        step = torch.exp2((torch.frexp(a).exponent - 4).clamp(min=-9).float())
        scale = torch.where(most > 0, (torch.round(a / step) * step).clamp(2.0 ** -9, 448.0), 0.0)
        y = x * unit[..., None] / torch.where(scale > 0, scale, 1.0)[..., None]
    y = y.clamp(-6.0, 6.0)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return torch.round(y / step) * step, scale, e


def values(x, fmt):
    """What x stands for after quantisation, in 32 bits."""
    y, scale, e = scaled_blocks(x, fmt)
    return (y * (scale * torch.exp2(e.float())[:, None])[..., None]).view(x.shape[0], -1)[:, : x.shape[1]]


def stored(x, fmt):
    """x in 4-bit form as a program holds it: codes, tiled scales, row exponents (nvfp4), rows and k."""
    rows, k = x.shape
    y, scale, e = scaled_blocks(x, fmt)
    a = y.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    code = torch.nn.functional.pad(code.view(rows, -1)[:, :k], (0, -k % 32))
    codes = code[:, 0::2] | code[:, 1::2] << 4
    m, ex = torch.frexp(scale)
    if fmt == "mxfp4":
        byte = torch.where(scale > 0, ex + 126, 0)
    else:  # E4M3: subnormals count in steps of 2^-9
        byte = torch.where(scale < 2.0 ** -6, scale * 512, (ex + 6) * 8 + (m * 16 - 8))
    byte = torch.nn.functional.pad(byte.to(torch.uint8), (0, -scale.shape[1] % (256 // FORMATS[fmt]), 0, -rows % 128))
    tiles = byte.view(byte.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return {"codes": codes.contiguous(), "scales": tiles, "exponents": e if fmt == "nvfp4" else None, "rows": rows, "k": k, "fmt": fmt}


def unpacked(q, dtype=torch.float32):
    """The codes' values, the scales and the rows' powers of two of a stored matrix: (rows, blocks, size), (rows, blocks, 1), (rows, 1)."""
    rows, k, fmt = q["rows"], q["k"], q["fmt"]
    size = FORMATS[fmt]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=dtype)
    code = torch.stack((q["codes"] & 15, q["codes"] >> 4), 2).view(rows, -1)
    code = torch.nn.functional.pad(code[:, :k], (0, -k % size)).view(rows, -1, size)
    v = table[(code & 7).long()] * (1 - 2 * (code >> 3).to(dtype))
    chunks = -(-k // 256) * (64 // size)
    byte = q["scales"].view(-1, chunks, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, chunks * 4)[:rows, : code.shape[1]].to(dtype)
    if fmt == "mxfp4":
        return v, torch.exp2(byte - 127)[..., None], torch.ones(rows, 1, device="cuda", dtype=dtype)
    m, ex = byte % 8, torch.floor(byte / 8)
    scale = torch.where(ex > 0, (8 + m) * torch.exp2(ex - 10), m * 2.0 ** -9)
    return v, scale[..., None], torch.exp2(q["exponents"].to(dtype))[:, None]


def stood_for(q, dtype=torch.float32):
    v, scale, row = unpacked(q, dtype)
    return (v * scale).view(q["rows"], -1)[:, : q["k"]] * row


def served(s, dtype):
    """The three matrices of a 4-bit block."""
    pair = stood_for(s["w_in"], dtype).view(-1, 2, 32, s["d"])
    return pair[:, 0].reshape(-1, s["d"])[: s["f"]], pair[:, 1].reshape(-1, s["d"])[: s["f"]], stood_for(s["w_out"], dtype)


# ---- one pass --------------------------------------------------------------

def activation(g, act):
    """act(g) and its derivative, in g's precision."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k, a = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (g + a * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * a * g * g)


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import extended_precision_gemm_gb300 as ddg

    kind = s["kind"]
    if kind == "quantise":
        return ddg.mx4_dequantize(ddg.mx4_quantize(s["x"], s["fmt"], cols=s["cols"]), torch.bfloat16)
    if kind == "product":
        return ddg.mx4_gemm(ddg.MX4(**s["a"]), ddg.MX4(**s["b"]), dtype=TYPES[s["type"]])
    if kind == "serve":
        return ddg.mx4_ff_gated(s["x"], ddg.MX4(**s["w_in"]), ddg.MX4(**s["w_out"]), act=s["act"])
    if kind == "forward":
        return ddg.ff_gated(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"])
    y, saved = ddg.ff_gated(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"], save=True)
    dx, dwg, dwu, dwd = ddg.ff_gated_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], saved)
    return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}


def run_plain(s):
    kind = s["kind"]
    if kind == "quantise":
        return values(s["x"].t() if s["cols"] else s["x"], s["fmt"]).to(torch.bfloat16)
    if kind == "product":
        return (stood_for(s["a"]) @ stood_for(s["b"]).t()).to(TYPES[s["type"]])
    dtype = TYPES[s["type"]]
    x = s["x"].float()
    if kind == "serve":
        x = values(x, s["fmt"])
        wg, wu, wd = served(s, torch.float32)
        h = values(activation(x @ wg.t(), s["act"])[0] * (x @ wu.t()), s["fmt"])
        return (h @ wd.t()).to(dtype)
    wg, wu, wd = (s[n].float() for n in ("wg", "wu", "wd"))
    u = x @ wu.t()
    a, da = activation(x @ wg.t(), s["act"])
    y = ((a * u) @ wd.t()).to(dtype)
    if kind == "forward":
        return y
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    grads = {"dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x, "dwd": dy.t() @ (a * u)}
    return {"y": y, **{n: v.to(dtype) for n, v in grads.items()}}


# ---- the definition in 64 bits ---------------------------------------------

def nearest(x, fmt):
    """x (rows, k) in 64 bits after quantisation: each block against the list of codes."""
    rows, k = x.shape
    size = FORMATS[fmt]
    x = torch.cat((x.double(), torch.zeros(rows, -k % size, dtype=torch.float64, device=x.device)), 1).reshape(rows, -1, size)
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


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantise":
        return nearest(s["x"].mT if case["cols"] else s["x"], case["fmt"])
    if kind == "product":
        return torch.einsum("mk,nk->mn", stood_for(s["a"], torch.float64), stood_for(s["b"], torch.float64))
    x = s["x"].double()
    if kind == "serve":
        x = nearest(x, case["fmt"])
        wg, wu, wd = served(s, torch.float64)
    else:
        wg, wu, wd = (s[n].double() for n in ("wg", "wu", "wd"))
    g, u = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
    if case["act"] == "silu":
        p = torch.sigmoid(g)
        slope = p + g * p * (1 - p)
    elif case["act"] == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        slope = p + g * torch.exp(-g * g / 2) * (0.5 / math.pi) ** 0.5
    elif case["act"] == "gelu_tanh":  # (1 + tanh z) / 2 = sigmoid(2 z)
        z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        p = torch.sigmoid(z)
        slope = p + g * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    else:
        p = slope = torch.heaviside(g, torch.zeros_like(g))
    h = g * p * u
    if kind == "serve":
        return torch.einsum("tf,df->td", nearest(h, case["fmt"]), wd)
    y = torch.einsum("tf,df->td", h, wd)
    if kind == "forward":
        return y
    dy = s["dy"].double()
    dh = torch.einsum("td,df->tf", dy, wd)
    dg, du = dh * u * slope, dh * g * p
    return {"y": y, "dx": torch.einsum("tf,fd->td", dg, wg) + torch.einsum("tf,fd->td", du, wu), "dwg": torch.einsum("tf,td->fd", dg, x),
            "dwu": torch.einsum("tf,td->fd", du, x), "dwd": torch.einsum("td,tf->df", dy, h)}
