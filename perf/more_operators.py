"""Cases of the operators around a layer's linear products in a training step, their plain forms and their 64-bit definitions.

What a transformer's training step computes between the gradients' partition
and its 4-bit products: the residual stream, and linear layers in 8 bits.

  embed       rows of a 16-bit table by token, times a factor; an id outside
              the table is padding and gives zeros
  embed_grad  the table's gradient: every row is the factor times the sum of
              the gradients of its tokens, 0 where no token names it
  dropout     elements dropped by a counter-based generator (Philox4x32-10,
              Salmon et al. 2011): the same call is its own backward pass
  norm        residual + dropped branch, rounded to 16 bits: the new stream;
              its root-mean-square norm in 16 bits, and in microscaled 8 or 4
              bits (which are read back)
  norm_grad   the gradients of the stream, of the branch and of the weight
  linear      16-bit activations quantised to microscaled 8 bits (e4m3 values,
              one power-of-two scale per 32) and multiplied with a weight
              that is held in them

``own`` False computes them with elementary torch operations in 32 bits;
True makes the library's calls.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
#: The magnitudes of e2m1's eight codes (the ninth bit pattern on is the sign).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: The largest exponent of the elements: what a block's scale leaves below its largest magnitude.
TOP = {4: 2, 8: 8}
#: Philox4x32: multipliers, and the key's increments (Salmon, Moraes, Dror, Shaw: Parallel random numbers, SC 2011).
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
OFFSET = 7   # the generator's stream of this layer and step


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call: one token of GPT-2 small, where launch and latency are all there is
        {"name": "embed_token", "op": "embed", "dtype": "bf16", "vocab": 50257, "dim": 768, "tokens": 1},
        # a rank's batch of 8 sequences of 1024 tokens through GPT-2 small's embedding, backward
        {"name": "embed_grad_gpt2", "op": "embed_grad", "dtype": "bf16", "vocab": 50257, "dim": 768, "tokens": 8192},
        # odd sizes in fp16: rows that start between vectors, padding among the tokens
        {"name": "embed_grad_ragged", "op": "embed_grad", "dtype": "fp16", "vocab": 32003, "dim": 1003, "tokens": 6007},
        # dropout of a ragged activation in fp16
        {"name": "dropout_ragged", "op": "dropout", "dtype": "fp16", "rows": 2047, "cols": 1003, "p": 0.25},
        # a training batch's residual branch of Llama-7B's width
        {"name": "dropout_batch", "op": "dropout", "dtype": "bf16", "rows": 8192, "cols": 4096, "p": 0.1},
        # one token at Llama-7B's width into the 8 bits that the next product reads
        {"name": "norm_token", "op": "norm", "dtype": "bf16", "rows": 1, "cols": 4096, "residual": True, "p": 0.0,
         "bits": 8, "wide": False},
        # a training batch: addition, dropout and norm, in 16 bits for the backward pass and in 8 for the product
        {"name": "norm_batch", "op": "norm", "dtype": "bf16", "rows": 8192, "cols": 4096, "residual": True, "p": 0.1,
         "bits": 8, "wide": True},
        # odd rows in fp16, no residual, 16 bits only
        {"name": "norm_ragged", "op": "norm", "dtype": "fp16", "rows": 1531, "cols": 1003, "residual": False, "p": 0.0,
         "bits": 0, "wide": True},
        # the backward pass of norm_batch
        {"name": "norm_grad_batch", "op": "norm_grad", "dtype": "bf16", "rows": 8192, "cols": 4096, "residual": True, "p": 0.1},
        # odd rows backward in fp16, without dropout
        {"name": "norm_grad_ragged", "op": "norm_grad", "dtype": "fp16", "rows": 2047, "cols": 1003, "residual": True, "p": 0.0},
        # one token through a Llama-7B MLP projection
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "tokens": 1, "inner": 4096, "outer": 11008},
        # a training batch through the same projection
        {"name": "linear_batch", "op": "linear", "dtype": "bf16", "tokens": 8192, "inner": 4096, "outer": 11008},
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm; about half are odd."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "embed_grad", "dropout", "norm", "norm", "norm_grad", "linear"))
    case = {"op": op, "dtype": rng.choice(("bf16", "fp16"))}
    if op in ("embed", "embed_grad"):
        case["vocab"], case["dim"] = _log(rng, 200, 60000), _log(rng, 64, 4500)
        case["tokens"] = _log(rng, 1, 20000)
    elif op == "linear":
        case["tokens"] = _log(rng, 1, 6000)
        case["inner"], case["outer"] = _log(rng, 100, 6000), _log(rng, 100, 9000)
    else:
        case["rows"], case["cols"] = _log(rng, 1, 8000), _log(rng, 64, 8300)
        case["p"] = rng.choice((0.1, 0.25, 0.5)) if op == "dropout" else rng.choice((0.0, 0.1, 0.25))
        if op != "dropout":
            case["residual"] = rng.choice((True, True, False))
        if op == "norm":
            case["bits"] = rng.choice((0, 4, 8, 8))
            case["wide"] = case["bits"] == 0 or rng.choice((True, False))
    return case


def work(case):
    if case["op"] == "embed":        # a row in and a row out for every token
        return {"bytes": case["tokens"] * (4 * case["dim"] + 8), "flops": case["tokens"] * case["dim"]}
    if case["op"] == "embed_grad":   # the tokens' gradients in, the whole table's out
        t, d = case["tokens"], case["dim"]
        return {"bytes": t * (2 * d + 8) + case["vocab"] * 2 * d, "flops": t * d}
    if case["op"] == "linear":
        t, k, n = case["tokens"], case["inner"], case["outer"]
        return {"bytes": int(2 * t * k + n * k * (1 + 1 / 32) + 2 * t * n), "flops": 2 * t * k * n}
    n = case["rows"] * case["cols"]
    if case["op"] == "dropout":
        return {"bytes": 4 * n, "flops": n}
    if case["op"] == "norm_grad":    # the output's gradient and the stream in (and the stream's gradient); theirs out
        return {"bytes": n * (4 + 2 + (2 if case["residual"] else 0) + (2 if case["p"] else 0)) + 4 * case["cols"], "flops": 12 * n}
    q = case["bits"] / 8 + 1 / 32 if case["bits"] else 0
    more = case["residual"] or case["p"] > 0     # then the stream is written too
    return {"bytes": int(n * (2 + (2 if case["residual"] else 0) + (2 if more else 0) + (2 if case["wide"] else 0)
                              + (2 * q + 2 if q else 0))) + 2 * case["cols"], "flops": 6 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g):
    """Normal, with rows of unlike size and a few channels that are many times larger."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    return x * (1 + 15 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01).float())


def _tiles(rows, cols):
    """The scale tiles of a matrix: 128 rows by 4 blocks of 32 columns each."""
    return (rows + 127) // 128, (cols + 127) // 128


def _codes_room(rows, cols, bits):
    """Codes (whole blocks of 32 a row) and scale tiles."""
    return (torch.empty(rows * ((cols + 31) // 32) * 4 * bits, dtype=torch.uint8, device="cuda"),
            torch.empty(512 * math.prod(_tiles(rows, cols)), dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = _gen(seed)
    td = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("embed", "embed_grad"):
        v, d, t = case["vocab"], case["dim"], case["tokens"]
        s["factor"] = math.sqrt(d)
        # by Zipf's law: the frequency of a token falls with its rank
        rank = torch.exp(torch.rand(t, generator=g, device="cuda", dtype=torch.float64) * math.log(v)).long() - 1
        s["ids"] = rank.clamp(0, v - 1) * 7919 % v
        if t % 2:      # an odd count: the batch has padding
            s["ids"][torch.rand(t, generator=g, device="cuda") < 0.05] = -1
        if case["op"] == "embed":
            s["table"] = (0.02 * torch.randn((v, d), generator=g, device="cuda")).to(td)
            s["out"] = torch.empty((t, d), dtype=td, device="cuda")
        else:
            s["grad"] = (1e-3 * torch.randn((t, d), generator=g, device="cuda")).to(td)
            s["out"] = torch.empty((v, d), dtype=td, device="cuda")
            # a bound on the library's scratch that a program without the library can state too
            s["workspace"] = torch.empty(t * (24 + d) + (1 << 20), dtype=torch.uint8, device="cuda")
    elif case["op"] == "linear":
        t, k, n = case["tokens"], case["inner"], case["outer"]
        s["x"] = _activations(t, k, g).to(td)
        codes, exps = _codes8(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
        s["w_codes"] = codes.reshape(-1).contiguous()
        rt, kt = _tiles(n, k)
        tiled = torch.zeros((rt * 128, kt * 4), dtype=torch.uint8, device="cuda")
        tiled[:n, :exps.shape[1]] = exps
        s["w_scales"] = tiled.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()
        s["x_codes"], s["x_scales"] = _codes_room(t, k, 8)
        s["y"] = torch.empty((t, n), dtype=td, device="cuda")
    else:
        rows, cols = case["rows"], case["cols"]
        s["seed"] = seed * 1000003 + 12345
        s["out"] = torch.empty((rows, cols), dtype=td, device="cuda")
        if case["op"] == "dropout":
            s["x"] = _activations(rows, cols, g).to(td)
            return s
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(td)
        stream = _activations(rows, cols, g)
        if case["op"] == "norm":
            s["x"] = torch.randn((rows, cols), generator=g, device="cuda").to(td) if case["residual"] else stream.to(td)
            s["res"] = stream.to(td) if case["residual"] else None
            s["h"] = torch.empty((rows, cols), dtype=td, device="cuda") if case["residual"] or case["p"] else None
            if case["bits"]:
                s["codes"], s["scales"] = _codes_room(rows, cols, case["bits"])
                s["values"] = torch.empty((rows, cols), dtype=td, device="cuda")
        else:
            s["h"] = stream.to(td)
            s["dy"] = (1e-2 * torch.randn((rows, cols), generator=g, device="cuda")).to(td)
            s["dh"] = (1e-2 * torch.randn((rows, cols), generator=g, device="cuda")).to(td) if case["residual"] else None
            s["dx"] = torch.empty((rows, cols), dtype=td, device="cuda") if case["p"] else None
            s["dw"] = torch.empty(cols, dtype=td, device="cuda")
            s["workspace"] = torch.empty(4 * 2048 * cols, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _keep(s):
    """Which elements a dropout keeps, [rows, cols], and the factor of those: 16 bits of the generator for each,
    those of a row's 8 consecutive columns from one counter."""
    rows, cols = s["rows"], s["cols"]
    groups = (cols + 7) // 8
    n = torch.arange(rows * groups, device="cuda")                # the counter: 4 words, least first
    x0, x1 = n & 0xFFFFFFFF, n >> 32
    x2, x3 = torch.full_like(n, OFFSET), torch.zeros_like(n)
    k0, k1 = s["seed"] & 0xFFFFFFFF, s["seed"] >> 32 & 0xFFFFFFFF
    for _ in range(10):
        a, b = PHILOX_M[0] * x0, PHILOX_M[1] * x2                 # 64 bits each, the sign bit among them
        x0, x1, x2, x3 = (b >> 32 & 0xFFFFFFFF) ^ x1 ^ k0, b & 0xFFFFFFFF, (a >> 32 & 0xFFFFFFFF) ^ x3 ^ k1, a & 0xFFFFFFFF
        k0, k1 = k0 + PHILOX_W[0] & 0xFFFFFFFF, k1 + PHILOX_W[1] & 0xFFFFFFFF
    words = torch.stack((x0, x1, x2, x3), 1)
    halves = torch.stack((words & 0xFFFF, words >> 16), 2).view(rows, groups * 8)[:, :cols]
    drop = round(s["p"] * 65536)
    return halves >= drop, 65536 / (65536 - drop)


def _dropped(x, s):
    """x (fp32) with its dropout."""
    if not s["p"]:
        return x
    keep, factor = _keep(s)
    return torch.where(keep, x * factor, 0.0)


def _scaled(x, bits):
    """x [rows, cols] (fp32) in blocks over its blocks' scales, [rows, blocks, 32], and the scales' exponents."""
    b = torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).view(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    _, e = torch.frexp(top)                        # |x| < 2^e, so the leading bit has the weight 2^(e-1)
    e = torch.where(top > 0, e - 1 - TOP[bits], -127).clamp(-127, 127)
    return torch.ldexp(b, -e.unsqueeze(2)), e


def _codes8(x):
    """Codes [rows, padded cols] and scale bytes [rows, blocks] of x in microscaled 8 bits."""
    y, e = _scaled(x.float(), 8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1), (e + 127).to(torch.uint8)


def _values8(codes, exps):
    """What codes and scale bytes stand for, in fp32."""
    v = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    return torch.ldexp(v, exps.to(torch.int32).unsqueeze(2) - 127).flatten(1)


def _mx_values(x, bits):
    """x (fp32) as microscaled 8 or 4 bits hold it."""
    if bits == 8:
        return _values8(*_codes8(x))[:, :x.shape[1]]
    y, e = _scaled(x, 4)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    v = torch.copysign(torch.tensor(E2M1, device="cuda")[code.long()], y)
    return torch.ldexp(v, e.unsqueeze(2)).flatten(1)[:, :x.shape[1]]


def _plain(s):
    td = DTYPES[s["dtype"]]
    if s["op"] == "embed":
        rows = s["table"][s["ids"].clamp(0, s["vocab"] - 1)].float() * s["factor"]
        return s["out"].copy_(torch.where((s["ids"] >= 0).unsqueeze(1), rows, 0.0))
    if s["op"] == "embed_grad":
        at = torch.where(s["ids"] >= 0, s["ids"], s["vocab"])     # padding goes to a row of its own
        sums = torch.zeros((s["vocab"] + 1, s["dim"]), device="cuda").index_add_(0, at, s["grad"].float())
        return s["out"].copy_(sums[:-1] * s["factor"])
    if s["op"] == "dropout":
        return s["out"].copy_(_dropped(s["x"].float(), s))
    if s["op"] == "norm":
        h, outs = s["x"], {}
        if s["h"] is not None:
            h = _dropped(s["x"].float(), s)
            h = outs["h"] = s["h"].copy_(h + s["res"].float() if s["residual"] else h)
        h = h.float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
        if s["wide"]:
            outs["y"] = s["out"].copy_(y)
        if s["bits"]:
            outs["values"] = s["values"].copy_(_mx_values(y, s["bits"]))
        return outs
    if s["op"] == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        g = dy * s["weight"].float()
        dh = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
        if s["residual"]:
            dh = dh + s["dh"].float()
        outs = {"dh": s["out"].copy_(dh), "dw": s["dw"].copy_((dy * h * r).sum(0))}
        if s["p"]:
            outs["dx"] = s["dx"].copy_(_dropped(dh, s))
        return outs
    k, n = s["inner"], s["outer"]
    x = _values8(*_codes8(s["x"]))[:, :k]
    rt, kt = _tiles(n, k)
    exps = s["w_scales"].view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    w = _values8(s["w_codes"].view(n, -1), exps[:n, :(k + 31) // 32])[:, :k]
    return s["y"].copy_(x @ w.t())


# ---------------------------------------------------------- library's calls
def _library(s):
    import zero_partitioned_mixed_gb300 as Z

    dt = Z.ZERO_BF16 if s["dtype"] == "bf16" else Z.ZERO_FP16
    if s["op"] == "embed":
        Z.zero_embedding(dt, s["vocab"], s["dim"], s["table"], s["tokens"], s["ids"], s["out"], scale=s["factor"])
        return s["out"]
    if s["op"] == "embed_grad":
        Z.zero_embedding_backward(dt, s["vocab"], s["dim"], s["grad"], s["tokens"], s["ids"], s["out"], s["workspace"],
                                  scale=s["factor"])
        return s["out"]
    if s["op"] == "linear":
        t, k, n = s["tokens"], s["inner"], s["outer"]
        Z.zero_mx8_quantize(dt, t, k, s["x"], s["x_codes"], s["x_scales"])
        Z.zero_mx8_matmul(dt, t, n, k, s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["y"])
        return s["y"]
    rows, cols = s["rows"], s["cols"]
    drop = Z.dropout_spec(s["p"], s["seed"], OFFSET) if s["p"] else None
    if s["op"] == "dropout":
        Z.zero_dropout(dt, rows, cols, s["x"], s["out"], drop)
        return s["out"]
    if s["op"] == "norm":
        outs = {} if s["h"] is None else {"h": s["h"]}
        Z.zero_rms_norm(dt, rows, cols, s["x"], s["weight"], EPS, residual16=s["res"], h16=s["h"],
                        out16=s["out"] if s["wide"] else None, bits=s["bits"], codes=s.get("codes"),
                        scales=s.get("scales"), dropout=drop)
        if s["wide"]:
            outs["y"] = s["out"]
        if s["bits"]:
            back = Z.zero_mx8_dequantize if s["bits"] == 8 else Z.zero_mx4_dequantize
            back(dt, rows, cols, s["codes"], s["scales"], s["values"])
            outs["values"] = s["values"]
        return outs
    Z.zero_rms_norm_backward(dt, rows, cols, s["dy"], s["h"], s["weight"], EPS, s["out"], s["workspace"],
                             dh_in16=s["dh"], dx16=s["dx"], dweight16=s["dw"], dropout=drop)
    outs = {"dh": s["out"], "dw": s["dw"]}
    if s["p"]:
        outs["dx"] = s["dx"]
    return outs


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------- definitions in 64 bits
def _philox_exact(seed, stream, groups):
    """The generator's 8 halves for every counter 0..groups-1: numpy, whole numbers of 64 bits."""
    low = np.uint64(0xFFFFFFFF)
    n = np.arange(groups, dtype=np.uint64)
    c = [n & low, n >> np.uint64(32), np.full_like(n, stream), np.zeros_like(n)]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for step in range(10):
        hi_lo = [(p >> np.uint64(32), p & low) for p in (c[0] * np.uint64(PHILOX_M[0]), c[2] * np.uint64(PHILOX_M[1]))]
        k = [np.uint64((key[i] + step * PHILOX_W[i]) % 2 ** 32) for i in (0, 1)]
        c = [hi_lo[1][0] ^ c[1] ^ k[0], hi_lo[1][1], hi_lo[0][0] ^ c[3] ^ k[1], hi_lo[0][1]]
    return np.stack([w >> np.uint64(16 * h) & np.uint64(0xFFFF) for w in c for h in (0, 1)], 1)


def _multiplier(s):
    """0 for a dropped element and 1 / (1 - share dropped) for a kept one, float64."""
    rows, cols, drop = s["rows"], s["cols"], int(s["p"] * 65536 + 0.5)
    halves = _philox_exact(s["seed"], OFFSET, rows * ((cols + 7) // 8)).reshape(rows, -1)[:, :cols]
    return torch.from_numpy((halves >= drop).astype(np.float32)).cuda().double() / (1 - drop / 65536)


def _nearest(a, bits):
    """Every magnitude (float64) at the nearest that the element type holds, ties to the even one, saturating."""
    if bits == 4:
        expo, low, top, digits = torch.floor(torch.log2(a.clamp(min=1e-300))), 0, 6.0, 1
    else:
        expo, low, top, digits = torch.floor(torch.log2(a.clamp(min=1e-300))), -6, 448.0, 3
    step = torch.exp2(expo.clamp(min=low) - digits)
    return (torch.round(a / step) * step).clamp(max=top)


def _mx_exact(x, bits):
    """x (float64, [rows, cols]) after microscaled rounding along its rows: the scale of a block is
    2^(floor(log2(largest magnitude)) - the element type's largest exponent)."""
    cols = x.shape[1]
    b = torch.cat((x, x.new_zeros((x.shape[0], -cols % 32))), 1).unflatten(1, (-1, 32))
    top = b.abs().amax(2, keepdim=True)
    expo = torch.floor(torch.log2(top))
    expo = expo - (torch.exp2(expo) > top).double() + (torch.exp2(expo + 1) <= top).double()
    scale = torch.where(top > 0, torch.exp2((expo - TOP[bits]).clamp(min=-127.0)), torch.ones_like(top))
    return (torch.copysign(_nearest((b / scale).abs(), bits), b) * scale).flatten(1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    td = DTYPES[case["dtype"]]
    if case["op"] == "embed":
        out = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device="cuda")
        real = torch.nonzero(s["ids"] >= 0).flatten()
        out[real] = s["table"][s["ids"][real]].double() * s["factor"]
        return out
    if case["op"] == "embed_grad":
        out = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        real = torch.nonzero(s["ids"] >= 0).flatten()
        return out.index_put_((s["ids"][real],), s["grad"][real].double() * s["factor"], accumulate=True)
    if case["op"] == "dropout":
        return s["x"].double() * _multiplier(s)
    if case["op"] == "norm":
        outs, h = {}, s["x"].double()
        if s["h"] is not None:
            if case["p"]:
                h = h * _multiplier(s)
            if case["residual"]:
                h = h + s["res"].double()
            outs["h"] = h
            h = h.to(td).double()                  # the norm is that of the stream as it is stored
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].double()
        if case["wide"]:
            outs["y"] = y
        if case["bits"]:
            outs["values"] = _mx_exact(y, case["bits"])
        return outs
    if case["op"] == "norm_grad":
        h, dy = s["h"].double(), s["dy"].double()
        unit = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        g = dy * s["weight"].double()
        # y = w h/rms: the part of g along h does not change it, but for eps
        dh = (g - unit * (g * unit).mean(1, keepdim=True)) / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        if case["residual"]:
            dh = dh + s["dh"].double()
        outs = {"dh": dh, "dw": (dy * unit).sum(0)}
        if case["p"]:
            outs["dx"] = dh * _multiplier(s)
        return outs
    t, k, n = case["tokens"], case["inner"], case["outer"]
    code = s["w_codes"].view(n, -1)[:, :k].long()
    expo, digits = code >> 3 & 15, (code & 7).double()
    magnitude = torch.where(expo > 0, (8 + digits) * torch.exp2(expo.double() - 10), digits * 2.0 ** -9)
    row = torch.arange(n, device="cuda").unsqueeze(1)
    block = torch.arange(k, device="cuda").unsqueeze(0) // 32
    # the byte of (row, block): tiles of 128 x 4 in row-major order; in a tile 32 lines of 4 row groups of 4 blocks
    at = ((row // 128 * ((k + 127) // 128) + block // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + block % 4)
    w = torch.where(code > 127, -magnitude, magnitude) * torch.exp2(s["w_scales"][at].double() - 127)
    return _mx_exact(s["x"].double(), 8) @ w.t()
