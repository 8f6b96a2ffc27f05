"""Cases of the matrix-optimizer and 4-bit operators, their plain forms and their 64-bit definitions.

Four paths of a partitioned training step whose hidden matrices are updated
by orthogonalised momentum, with the weights then exchanged in 4 bits:

  momentum  the ranks' 16-bit gradients of a flat region are averaged and
            unscaled, the fp32 momentum advances, the (Nesterov) update is
            rounded to bf16
  ortho     a batch of matrices is orthogonalised by the quintic
            Newton-Schulz iteration, its result rounded to bf16
  apply     decoupled weight decay and the orthogonalised update on the fp32
            master, rounded into every rank's 16-bit replica
  mx4       a matrix is quantised to microscaled 4-bit floats (e2m1 values,
            one power-of-two scale per 32) along its rows or its columns,
            and read back as 16-bit values
  linear    16-bit activations are quantised and multiplied with a weight
            that is held in microscaled 4 bits

``own`` False computes them with elementary torch operations in 32 bits;
True makes the library's calls.
"""

import math

import torch

own = False

#: Quintic coefficients of the Newton-Schulz iteration, and its steps.
NS_A, NS_B, NS_C, NS_STEPS = 3.4445, -4.7750, 2.0315, 5
LR, MU, DECAY = 0.02, 0.95, 0.1
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
#: The magnitudes of e2m1's eight codes (the ninth bit pattern on is the sign).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call: one small projection of a toy model, where launches and latency are all there is
        {"name": "ortho_small", "op": "ortho", "dtype": "bf16", "batch": 1, "rows": 96, "cols": 160},
        # GPT-2 small's attention output projections, all 12 layers in one call
        {"name": "ortho_gpt2_attn", "op": "ortho", "dtype": "bf16", "batch": 12, "rows": 768, "cols": 768},
        # odd and tall: neither size a multiple of a tile or of a vector, fp16
        {"name": "ortho_ragged", "op": "ortho", "dtype": "fp16", "batch": 6, "rows": 1531, "cols": 1003},
        # a Llama-7B MLP projection, the largest matrix of a layer
        {"name": "ortho_llama_mlp", "op": "ortho", "dtype": "bf16", "batch": 1, "rows": 11008, "cols": 4096},
        # an odd region of a few layers of a small model on 4 ranks
        {"name": "momentum_odd", "op": "momentum", "dtype": "fp16", "ranks": 4, "count": 1000003},
        # every hidden matrix of GPT-2 small on 8 ranks
        {"name": "momentum_gpt2", "op": "momentum", "dtype": "bf16", "ranks": 8, "count": 84934656},
        # the toy GPT's flat buffer on 32 ranks: many replicas of little data
        {"name": "apply_toy", "op": "apply", "dtype": "fp16", "ranks": 32, "count": 637824},
        # the matrices of one Llama-7B layer on 8 ranks
        {"name": "apply_llama", "op": "apply", "dtype": "bf16", "ranks": 8, "count": 202375168},
        # a Llama-7B MLP weight quantised along its rows, as its forward product takes it
        {"name": "mx4_llama_mlp", "op": "mx4", "dtype": "bf16", "rows": 11008, "cols": 4096, "transpose": False},
        # a ragged weight quantised along its columns, as its backward product takes it
        {"name": "mx4_columns_ragged", "op": "mx4", "dtype": "fp16", "rows": 2047, "cols": 5003, "transpose": True},
        # one token through a Llama-7B MLP projection
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "tokens": 1, "inner": 4096, "outer": 11008},
        # a training batch through the same projection
        {"name": "linear_batch", "op": "linear", "dtype": "bf16", "tokens": 8192, "inner": 4096, "outer": 11008},
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm; about half are odd."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ortho", "ortho", "momentum", "apply", "mx4", "linear"))
    case = {"op": op, "dtype": rng.choice(("bf16", "fp16"))}
    if op == "ortho":
        case["rows"], case["cols"] = _log(rng, 16, 6000), _log(rng, 16, 6000)
        lo, hi = sorted((case["rows"], case["cols"]))
        room = _ortho_flops(1, 4096, 11008) // (2 * _ortho_flops(1, lo, hi))
        case["batch"] = _log(rng, 1, max(1, min(16, room)))
    elif op in ("momentum", "apply"):
        case["ranks"] = rng.choice((1, 2, 3, 4, 5, 8, 13, 16, 32))
        case["count"] = _log(rng, 20000, min(84000000, 640000000 // case["ranks"]))
    elif op == "mx4":
        case["rows"], case["cols"] = _log(rng, 1, 8000), _log(rng, 64, 5600)
        case["transpose"] = rng.choice((False, True))
    else:
        case["tokens"] = _log(rng, 1, 6000)
        case["inner"], case["outer"] = _log(rng, 100, 6000), _log(rng, 100, 9000)
    return case


def _ortho_flops(batch, short, wide):
    """Three products a step; the two symmetric ones need half of their entries."""
    return batch * NS_STEPS * (3 * short * short * wide + short ** 3)


def work(case):
    if case["op"] == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        return {"bytes": 4 * case["batch"] * m * n, "flops": _ortho_flops(case["batch"], m, n)}
    if case["op"] == "momentum":   # N gradients and the momentum in, the momentum and the update out
        return {"bytes": case["count"] * (2 * case["ranks"] + 4 + 4 + 2), "flops": case["count"] * (case["ranks"] + 4)}
    if case["op"] == "apply":      # the master and the update in, the master and N replicas out
        return {"bytes": case["count"] * (4 + 2 + 4 + 2 * case["ranks"]), "flops": case["count"] * 3}
    if case["op"] == "mx4":        # 16 bits in; 4 bits and a byte per 32 out, in again; 16 bits out
        n = case["rows"] * case["cols"]
        return {"bytes": int(n * (2 + 2 * (0.5 + 1 / 32) + 2)), "flops": 3 * n}
    t, k, n = case["tokens"], case["inner"], case["outer"]
    return {"bytes": int(2 * t * k + n * k * (0.5 + 1 / 32) + 2 * t * n), "flops": 2 * t * k * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _gradient(shape, g):
    """A matrix gradient as training meets it: a few strong directions over noise."""
    batch, rows, cols = shape
    r = max(1, min(rows, cols) // 8)
    u = torch.randn((batch, rows, r), generator=g, device="cuda")
    v = torch.randn((batch, r, cols), generator=g, device="cuda")
    return 1e-3 * (torch.bmm(u, v) / math.sqrt(r) + 0.3 * torch.randn(shape, generator=g, device="cuda"))


def _pitch(cols):
    """Bytes of one row of codes: whole blocks of 32 values."""
    return (cols + 31) // 32 * 16


def _tiles(rows, cols):
    """The scale tiles of a matrix: 128 rows by 4 blocks of 32 columns each."""
    return (rows + 127) // 128, (cols + 127) // 128


def prepare(case, seed):
    g = _gen(seed)
    td = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "ortho":
        shape = (case["batch"], case["rows"], case["cols"])
        s["src"] = _gradient(shape, g).to(td)
        s["dst"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")   # bf16 for both input types
        # a bound on the library's scratch that a program without the library can state too
        lo, hi = sorted(shape[1:])
        lo, hi = (lo + 63) // 64 * 64, (hi + 63) // 64 * 64
        s["workspace"] = torch.empty(case["batch"] * (4 * lo * hi + 10 * lo * lo + 65536) + (1 << 20),
                                     dtype=torch.uint8, device="cuda")
    elif case["op"] in ("momentum", "apply"):
        n, count = case["ranks"], case["count"]
        pad = (count + 7) // 8 * 8
        s["state"] = torch.zeros(16, dtype=torch.int32, device="cuda")
        s["state"].view(torch.float32)[0] = 1024.0 if case["op"] == "momentum" else 1.0   # the loss scale
        if case["op"] == "momentum":
            s["grads"] = torch.zeros((n, pad), dtype=td, device="cuda")
            for r in range(n):
                s["grads"][r, :count] = (1.024 * torch.randn(count, generator=g, device="cuda")).to(td)
            s["momentum"] = torch.zeros((2, pad), device="cuda")
            s["momentum"][0, :count] = 5e-3 * torch.randn(count, generator=g, device="cuda")
            s["update"] = torch.zeros(pad, dtype=torch.bfloat16, device="cuda")
        else:
            s["ortho"] = torch.zeros(pad, dtype=torch.bfloat16, device="cuda")
            s["ortho"][:count] = 0.02 * torch.randn(count, generator=g, device="cuda")
            s["master"] = torch.zeros(pad, device="cuda")
            s["master"][:count] = 0.02 * torch.randn(count, generator=g, device="cuda")
            s["params"] = torch.zeros((n, pad), dtype=td, device="cuda")
            s["params"][:] = s["master"].to(td)
    elif case["op"] == "mx4":
        rows, cols = case["rows"], case["cols"]
        # weights: normal, with rows of unlike size
        w = torch.randn((rows, cols), generator=g, device="cuda")
        s["src"] = (0.02 * w * torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))).to(td)
        r, c = (cols, rows) if case["transpose"] else (rows, cols)
        s["codes"] = torch.empty(r * _pitch(c), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(512 * math.prod(_tiles(r, c)), dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty((r, c), dtype=td, device="cuda")
    else:
        t, k, n = case["tokens"], case["inner"], case["outer"]
        # activations: normal, with a few channels that are many times larger
        x = torch.randn((t, k), generator=g, device="cuda")
        x *= 1 + 15 * (torch.rand((1, k), generator=g, device="cuda") < 0.01).float()
        s["x"] = x.to(td)
        w = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
        codes, exps = _mx4_codes(w)
        flat = torch.zeros((n, 2 * _pitch(k)), dtype=torch.uint8, device="cuda")
        flat[:, :codes.shape[1]] = codes
        s["w_codes"] = (flat[:, 0::2] | flat[:, 1::2] << 4).reshape(-1).contiguous()
        rt, kt = _tiles(n, k)
        tiled = torch.zeros((rt * 128, kt * 4), dtype=torch.uint8, device="cuda")
        tiled[:n, :exps.shape[1]] = exps
        s["w_scales"] = tiled.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()
        s["x_codes"] = torch.empty(t * _pitch(k), dtype=torch.uint8, device="cuda")
        s["x_scales"] = torch.empty(512 * math.prod(_tiles(t, k)), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((t, n), dtype=td, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _mx4_blocks(x):
    """x [rows, cols] in fp32 with its rows filled with zeros to whole blocks: [rows, blocks, 32]."""
    rows, cols = x.shape
    return torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)


def _mx4_codes(x):
    """The 4-bit code of every value of x, [rows, padded cols], and each block's scale byte, [rows, blocks]."""
    b = _mx4_blocks(x.float())
    _, e = torch.frexp(b.abs().amax(2))            # |x| < 2^e, so the leading bit has the weight 2^(e-1)
    e = torch.where(b.abs().amax(2) > 0, e - 3, -127).clamp(-127, 127)
    y = torch.ldexp(b, -e.unsqueeze(2))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code | torch.signbit(y).to(torch.uint8) << 3).flatten(1), (e + 127).to(torch.uint8)


def _mx4_values(codes, exps):
    """What codes [rows, padded cols] and scale bytes [rows, blocks] stand for, in fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = table[codes.long()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, exps.to(torch.int32).unsqueeze(2) - 127).flatten(1)


def _plain(s):
    td = DTYPES[s["dtype"]]
    if s["op"] == "ortho":
        x = s["src"].float()
        x = x / torch.sqrt((x * x).sum((1, 2), keepdim=True))
        if s["rows"] > s["cols"]:
            x = x.transpose(1, 2)
        for _ in range(NS_STEPS):
            a = torch.bmm(x, x.transpose(1, 2))
            x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
        return s["dst"].copy_(x.transpose(1, 2) if s["rows"] > s["cols"] else x)
    count = s.get("count", 0)
    if s["op"] == "momentum":
        g = s["grads"][:, :count].float().sum(0) / (s["ranks"] * s["state"].view(torch.float32)[0])
        m = MU * s["momentum"][0, :count] + g
        s["momentum"][1, :count] = m
        s["update"][:count] = g + MU * m
        return {"momentum": s["momentum"][1, :count], "update": s["update"][:count]}
    if s["op"] == "apply":
        p = (1 - LR * DECAY) * s["master"][:count] - LR * s["ortho"][:count].float()
        s["master"][:count] = p
        s["params"][:, :count] = p.to(td)
        return {"master": s["master"][:count], "params": s["params"][:, :count]}
    if s["op"] == "mx4":
        x = s["src"].t() if s["transpose"] else s["src"]
        return s["values"].copy_(_mx4_values(*_mx4_codes(x))[:, :x.shape[1]])
    k, n = s["inner"], s["outer"]
    x = _mx4_values(*_mx4_codes(s["x"]))[:, :k]
    w = s["w_codes"].view(n, -1)
    rt, kt = _tiles(n, k)
    exps = s["w_scales"].view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    w = _mx4_values(torch.stack((w & 15, w >> 4), 2).flatten(1), exps[:n, :(k + 31) // 32])[:, :k]
    return s["y"].copy_(x @ w.t())


# ---------------------------------------------------------- library's calls
def _library(s):
    import zero_partitioned_mixed_gb300 as Z

    dt = Z.ZERO_BF16 if s["dtype"] == "bf16" else Z.ZERO_FP16
    count = s.get("count", 0)
    if s["op"] == "ortho":
        Z.zero_orthogonalize(dt, s["rows"], s["cols"], s["src"].unbind(0), s["dst"].unbind(0), s["workspace"],
                             steps=NS_STEPS, coeffs=(NS_A, NS_B, NS_C))
        return s["dst"]
    if s["op"] == "momentum":
        Z.zero_muon_momentum(dt, count, s["grads"].unbind(0), s["momentum"], s["update"],
                             Z.muon_hyper(lr=LR, momentum=MU, weight_decay=DECAY), s["state"])
        return {"momentum": s["momentum"][1, :count], "update": s["update"][:count]}
    if s["op"] == "apply":
        Z.zero_muon_apply(dt, count, s["ortho"], s["master"], s["params"].unbind(0),
                          Z.muon_hyper(lr=LR, momentum=MU, weight_decay=DECAY), s["state"])
        return {"master": s["master"][:count], "params": s["params"][:, :count]}
    if s["op"] == "mx4":
        r, c = s["values"].shape
        Z.zero_mx4_quantize(dt, s["rows"], s["cols"], s["src"], s["codes"], s["scales"], transpose=s["transpose"])
        Z.zero_mx4_dequantize(dt, r, c, s["codes"], s["scales"], s["values"])
        return s["values"]
    t, k, n = s["tokens"], s["inner"], s["outer"]
    Z.zero_mx4_quantize(dt, t, k, s["x"], s["x_codes"], s["x_scales"])
    Z.zero_mx4_matmul(dt, t, n, k, s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["y"])
    return s["y"]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------- definitions in 64 bits
def _nearest_e2m1(v):
    """Every value of v (float64) at the nearest of e2m1's values, ties to the even code, saturating."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    a = v.abs().clamp(max=6.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=7)     # the first grid value >= a
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[take], v)


def _mx4_exact(x):
    """x (float64, [rows, cols]) after microscaled 4-bit rounding along its rows: the scale of a block
    is 2^(floor(log2(largest magnitude)) - 2), 2 being the largest exponent of e2m1."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    for at in range(0, cols, 32):
        block = x[:, at:at + 32]
        top = block.abs().amax(1, keepdim=True)
        expo = torch.floor(torch.log2(top))
        expo = expo - (torch.exp2(expo) > top).double() + (torch.exp2(expo + 1) <= top).double()
        scale = torch.where(top > 0, torch.exp2((expo - 2).clamp(min=-127.0)), torch.ones_like(top))
        out[:, at:at + 32] = _nearest_e2m1(block / scale) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        if case["batch"] * case["rows"] * case["cols"] * min(case["rows"], case["cols"]) > 3e11:
            return None
        out = torch.empty(s["src"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["batch"]):
            x = s["src"][i].double()
            x = x / torch.linalg.vector_norm(x)
            wide = case["rows"] <= case["cols"]
            for _ in range(NS_STEPS):
                # p(X) = X (a + b G + c G G) with the smaller of X's two Gram matrices
                gram = x @ x.t() if wide else x.t() @ x
                poly = NS_B * gram + NS_C * (gram @ gram)
                poly.diagonal().add_(NS_A)
                x = poly @ x if wide else x @ poly
            out[i] = x
        return out
    if case["op"] == "momentum":
        count, total = case["count"], torch.zeros(case["count"], dtype=torch.float64, device="cuda")
        for r in range(case["ranks"]):
            total += s["grads"][r, :count].double()
        total /= case["ranks"] * 1024.0
        m = torch.add(total, s["momentum"][0, :count].double(), alpha=MU)
        return {"momentum": m, "update": torch.add(total, m, alpha=MU)}
    if case["op"] == "apply":
        count = case["count"]
        p = s["master"][:count].double() * (1.0 - LR * DECAY)
        p.sub_(s["ortho"][:count].double(), alpha=LR)
        return {"master": p, "params": p.unsqueeze(0).expand(case["ranks"], count)}
    if case["op"] == "mx4":
        x = s["src"].double()
        return _mx4_exact(x.t().contiguous() if case["transpose"] else x)
    t, k, n = case["tokens"], case["inner"], case["outer"]
    low_high = s["w_codes"].view(n, -1, 1) >> torch.tensor([0, 4], dtype=torch.uint8, device="cuda") & 15
    code = low_high.reshape(n, -1)[:, :k].long()
    magnitude = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code & 7]
    row = torch.arange(n, device="cuda").unsqueeze(1)
    block = torch.arange(k, device="cuda").unsqueeze(0) // 32
    # the byte of (row, block): tiles of 128 x 4 in row-major order; in a tile 32 lines of 4 row groups of 4 blocks
    at = ((row // 128 * ((k + 127) // 128) + block // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + block % 4)
    scale = torch.exp2(s["w_scales"][at].double() - 127)
    w = torch.where(code > 7, -magnitude, magnitude) * scale
    return _mx4_exact(s["x"].double()) @ w.t()
