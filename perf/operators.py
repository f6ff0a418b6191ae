"""Cases of the E4M3 operators: the quantizer with a scale per block, the RMS norm and the gated activation that write
8-bit operands, and the products of such operands (one weight, and a stack of experts).

A tensor in 8 bits is a pair: codes (uint8, OCP E4M3 values) and float32 scales, one per block of 1 x 128
(activations) or 128 x 128 (weights); the last block of an axis may be short."""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # largest E4M3 value
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # The activations of a decode batch before a projection: a few rows, latency counts.
        {"name": "quantize_8x5120", "op": "quantize", "rows": 8, "k": 5120, "block_rows": 1},
        # A gate or up projection quantized when a checkpoint is loaded.
        {"name": "quantize_weight_17408x5120", "op": "quantize", "rows": 17408, "k": 5120, "block_rows": 128},
        # The norm before a projection in a decode batch.
        {"name": "norm_8x5120", "op": "norm", "rows": 8, "k": 5120, "residual": True},
        # The same in a prefill chunk.
        {"name": "norm_2048x5120", "op": "norm", "rows": 2048, "k": 5120, "residual": True},
        # Between gate/up and down of an MLP: decode batch, prefill chunk.
        {"name": "silu_8x17408", "op": "silu", "rows": 8, "n": 17408},
        {"name": "silu_2048x17408", "op": "silu", "rows": 2048, "n": 17408},
        # One token through a square projection.
        {"name": "linear_1x5120x5120", "op": "linear", "m": 1, "n": 5120, "k": 5120},
        # A decode batch through the up projection.
        {"name": "linear_32x17408x5120", "op": "linear", "m": 32, "n": 17408, "k": 5120},
        # The last, short chunk of a prompt through a projection whose sizes end inside a block on both axes.
        {"name": "linear_333x5000x17392", "op": "linear", "m": 333, "n": 5000, "k": 17392},
        # A prefill chunk through the up projection.
        {"name": "linear_2048x17408x5120", "op": "linear", "m": 2048, "n": 17408, "k": 5120},
        # A decode batch of a mixture-of-experts layer, and its prefill chunk.
        {"name": "grouped_8x8of128", "op": "grouped", "t": 8, "topk": 8, "experts": 128, "n": 2048, "k": 4096,
         "padded": 0},
        {"name": "grouped_2048x8of128", "op": "grouped", "t": 2048, "topk": 8, "experts": 128, "n": 2048, "k": 4096,
         "padded": 0},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "norm", "silu", "linear", "linear", "grouped"])
    # Half of the sizes end inside a block of 128, as a sharded or padded projection's do.
    step = rng.choice([16, 128])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 17408), "k": _log(rng, 128, 5120, step),
                "block_rows": rng.choice([1, 128])}
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 2048), "k": _log(rng, 128, 5120, step),
                "residual": rng.random() < 0.7}
    if op == "silu":
        return {"op": op, "rows": _log(rng, 1, 2048), "n": _log(rng, 128, 17408, step)}
    if op == "linear":
        n, k = _log(rng, 64, 17408, rng.choice([1, 8, 128])), _log(rng, 128, 17408, step)
        return {"op": op, "m": _log(rng, 1, min(2048, 2048 * 17408 * 5120 // (n * k))), "n": n, "k": k}
    experts = _log(rng, 4, 128)
    t = _log(rng, 1, 2048)
    return {"op": op, "t": t, "topk": rng.randint(1, min(8, experts)), "experts": experts,
            "n": _log(rng, 64, 2048, rng.choice([1, 8, 128])), "k": _log(rng, 128, 4096, step),
            "padded": rng.choice([0, t // 4])}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _blocks(x, block_rows):
    """[..., r, k] -> max |x| of each block, spread back to [..., r, k], and per block [..., rb, kb]."""
    r, k = x.shape[-2:]
    rb, kb = -(-r // block_rows), -(-k // BLOCK)
    p = torch.nn.functional.pad(x.abs(), (0, kb * BLOCK - k, 0, rb * block_rows - r))
    amax = p.reshape(*x.shape[:-2], rb, block_rows, kb, BLOCK).amax((-3, -1))
    return _spread(amax, block_rows, r, k), amax


def _spread(s, block_rows, r, k):
    return s.repeat_interleave(block_rows, -2)[..., :r, :].repeat_interleave(BLOCK, -1)[..., :k]


def _encode(v, block_rows):
    """Codes and scales; the quotients in 64 bits, since a value next to a border decides by its last bits."""
    amax, per_block = _blocks(v, block_rows)
    q = torch.where(amax > 0, v.double() * TOP / amax.double(), 0.0)
    return q.float().to(torch.float8_e4m3fn).view(torch.uint8), per_block.float() / TOP


def _decode(codes, scales, block_rows):
    r, k = codes.shape[-2:]
    return codes.view(torch.float8_e4m3fn).float() * _spread(scales, block_rows, r, k)


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _hidden(rows, k, gen):
    """Hidden states: standard normal, one channel in a hundred eight times as large."""
    x = _normal((rows, k), gen)
    x[:, torch.randperm(k, generator=gen, device="cuda")[:max(1, k // 100)]] *= 8
    return x.bfloat16()


def _route(case, gen):
    """Each token's distinct experts under a router that prefers some of them; padding tokens have id -1."""
    t, e = case["t"], case["experts"]
    logits = _normal((1, e), gen, 0.5) - torch.log(-torch.log(torch.rand((t, e), generator=gen, device="cuda")
                                                               .clamp_(1e-7, 1 - 1e-7)))
    route = logits.topk(case["topk"], dim=1).indices.to(torch.int32)
    if case["padded"]:
        route[t - case["padded"]:] = -1
    return route.contiguous()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], {"op": case["op"]}
    if op == "quantize":
        weight = case["block_rows"] != 1
        s["w"] = _normal((case["rows"], case["k"]), gen, 0.02).bfloat16() if weight \
            else _hidden(case["rows"], case["k"], gen)
        s["block_rows"] = case["block_rows"]
    elif op == "norm":
        s["x"] = _hidden(case["rows"], case["k"], gen)
        s["residual"] = (4 * _normal((case["rows"], case["k"]), gen)).bfloat16() if case["residual"] else None
        s["weight"] = (1 + _normal((case["k"],), gen, 0.1)).bfloat16()
    elif op == "silu":
        s["gate_up"] = _normal((case["rows"], 2 * case["n"]), gen, 2.0).bfloat16()
    elif op == "linear":
        s["xq"], s["xs"] = _encode(_hidden(case["m"], case["k"], gen), 1)
        s["wq"], s["ws"] = _encode(_normal((case["n"], case["k"]), gen, 0.02).bfloat16(), 128)
    else:
        s["xq"], s["xs"] = _encode(_hidden(case["t"], case["k"], gen), 1)
        pairs = [_encode(_normal((case["n"], case["k"]), gen, 0.02 * (1 + i / 64)).bfloat16(), 128)
                 for i in range(case["experts"])]
        s["wq"], s["ws"] = torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])
        s["route"] = _route(case, gen)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        import nvfp4_weight_only_amd as nv
        if op == "quantize":
            codes, scales = nv.fp8_quantize(s["w"], block_rows=s["block_rows"])
            return codes.view(torch.float8_e4m3fn), scales
        if op == "norm":
            codes, scales, h = nv.rmsnorm_fp8(s["x"], s["weight"], EPS, residual=s["residual"])
            return codes.view(torch.float8_e4m3fn), scales, h
        if op == "silu":
            codes, scales = nv.silu_mul_fp8(s["gate_up"])
            return codes.view(torch.float8_e4m3fn), scales
        if op == "linear":
            return nv.fp8_linear(s["xq"], s["xs"], s["wq"], s["ws"])
        return nv.fp8_linear_grouped(s["xq"], s["xs"], s["route"], s["wq"], s["ws"])
    if op == "quantize":
        codes, scales = _encode(s["w"].float(), s["block_rows"])
        return codes.view(torch.float8_e4m3fn), scales
    if op == "norm":
        # The sum is stored in 16 bits as the next layer's residual, and what is stored is what is normalized.
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).bfloat16()
        f = h.float()
        v = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        codes, scales = _encode(v, 1)
        return codes.view(torch.float8_e4m3fn), scales, None if s["residual"] is None else h
    if op == "silu":
        gate, up = s["gate_up"].float().chunk(2, -1)
        codes, scales = _encode(gate / (1 + torch.exp(-gate)) * up, 1)
        return codes.view(torch.float8_e4m3fn), scales
    if op == "linear":
        return (_decode(s["xq"], s["xs"], 1) @ _decode(s["wq"], s["ws"], 128).T).bfloat16()
    return _grouped(s)


def _grouped(s):
    x, route = _decode(s["xq"], s["xs"], 1), s["route"]
    (t, topk), e, n = route.shape, s["wq"].shape[0], s["wq"].shape[1]
    ids = route.reshape(-1).long()
    valid = (ids >= 0) & (ids < e)
    if t * topk <= e:  # few pairs: their experts' matrices alone
        at = torch.where(valid, ids, 0)
        y = (_decode(s["wq"][at], s["ws"][at], 128) @ x.repeat_interleave(topk, 0)[:, :, None])[:, :, 0]
        return torch.where(valid[:, None], y, 0.0).bfloat16().reshape(t, topk, n)
    # Many: the pairs sorted by expert, each expert's rows padded to the longest one's.
    key, order = torch.where(valid, ids, e).sort(stable=True)
    counts = torch.zeros(e + 1, dtype=torch.long, device=x.device).scatter_add_(0, key, torch.ones_like(key))
    slot = torch.arange(key.numel(), device=x.device) - (counts.cumsum(0) - counts)[key]
    cap = int(counts[:e].max())
    keep = key < e
    key, slot, order = key[keep], slot[keep], order[keep]
    rows = torch.zeros((e, cap, x.shape[1]), device=x.device)
    rows[key, slot] = x[order // topk]
    y = torch.zeros((t * topk, n), device=x.device)
    y[order] = (rows @ _decode(s["wq"], s["ws"], 128).transpose(1, 2))[key, slot]
    return y.bfloat16().reshape(t, topk, n)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        r, k = case["rows"], case["k"]
        return {"bytes": 3 * r * k + 4 * -(-r // case["block_rows"]) * -(-k // BLOCK), "flops": 2 * r * k}
    if op == "norm":
        r, k = case["rows"], case["k"]
        return {"bytes": (7 if case["residual"] else 3) * r * k + 4 * r * -(-k // BLOCK) + 2 * k, "flops": 6 * r * k}
    if op == "silu":
        r, n = case["rows"], case["n"]
        return {"bytes": 5 * r * n + 4 * r * -(-n // BLOCK), "flops": 8 * r * n}
    n, k = case["n"], case["k"]
    kb, nb = -(-k // BLOCK), -(-n // BLOCK)
    if op == "linear":
        m = case["m"]
        return {"bytes": m * k + 4 * m * kb + n * k + 4 * nb * kb + 2 * m * n, "flops": 2 * m * n * k}
    pairs, e = (case["t"] - case["padded"]) * case["topk"], case["experts"]
    used = e * (1 - (1 - 1 / e) ** pairs)  # experts that some pair chooses
    return {"bytes": case["t"] * (k + 4 * kb) + used * (n * k + 4 * nb * kb) + 4 * case["t"] * case["topk"]
            + 2 * case["t"] * case["topk"] * n, "flops": 2 * pairs * n * k}


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _e4m3_values(device):
    """The value of each of the 256 codes, from the format's fields: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    code = torch.arange(256, device=device)
    exp, man = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(exp > 0, (1 + man / 8) * torch.exp2((exp - 7).double()), man / 8 * 2.0 ** -6)
    mag[(exp == 15) & (man == 7)] = math.nan
    return torch.where(code >= 128, -mag, mag)


def _exact_blocks(v, block_rows):
    """(the values of the codes, the scales) of v [r, k] in 64 bits: each quotient to the nearest value of the grid."""
    r, k = v.shape
    scales = torch.empty((-(-r // block_rows), -(-k // BLOCK)), dtype=torch.float64, device=v.device)
    out = torch.empty_like(v)
    for b in range(scales.shape[1]):
        cols = v[:, b * BLOCK:(b + 1) * BLOCK]
        top = cols.abs().amax(1)
        top = torch.cat([top, top.new_zeros(scales.shape[0] * block_rows - r)]).reshape(-1, block_rows).amax(1)
        scales[:, b] = top / TOP
        top = top.repeat_interleave(block_rows)[:r, None]
        q = torch.where(top > 0, cols * TOP / top, torch.zeros_like(cols))
        # Below 2^-6 the grid's step is 2^-9, above it an eighth of the power of two; round() takes ties to even.
        step = torch.exp2(torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
        out[:, b * BLOCK:(b + 1) * BLOCK] = (q / step).round() * step
    return out, scales


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        return _exact_blocks(s["w"].double(), s["block_rows"])
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).bfloat16().double()
        # A row's factor cancels in the quotients, which are ratios of 16-bit products: with ties, which it would break.
        codes, scales = _exact_blocks(h * s["weight"].double(), 1)
        scales /= ((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS).sqrt()
        return codes, scales, None if s["residual"] is None else h
    if op == "silu":
        g, u = s["gate_up"].double().tensor_split(2, -1)
        return _exact_blocks(g * torch.sigmoid(g) * u, 1)
    table = _e4m3_values(s["xq"].device)

    def value(codes, scales, block_rows):
        v = table[codes.int()]
        for b in range(scales.shape[1]):
            v[:, b * BLOCK:(b + 1) * BLOCK] *= scales[:, b].double().repeat_interleave(block_rows)[:v.shape[0], None]
        return v

    x = value(s["xq"], s["xs"], 1)
    if op == "linear":
        return x @ value(s["wq"], s["ws"], 128).T
    (t, topk), (e, n, k) = s["route"].shape, s["wq"].shape
    y = torch.zeros((t * topk, n), dtype=torch.float64, device=x.device)
    ids = s["route"].reshape(-1)
    for i in range(e):
        at = (ids == i).nonzero()[:, 0]
        y[at] = x[at // topk] @ value(s["wq"][i], s["ws"][i], 128).T
    return y.reshape(t, topk, n)
