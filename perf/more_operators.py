"""Cases of the operators around a paged FP4 cache of keys and values: rotary positions, appending rows to the cache
(with the position rotation applied to the keys on the way), and attention that reads the cache.

A cache is one layer's keys and values in pages of block_size tokens: codes (uint8, two E2M1 values a byte, the even
element in the low nibble) [pages, block_size, heads, head_dim / 2] and a scale per 16 (format "nvfp4": E4M3, with an
FP32 tensor scale) or 32 elements ("mxfp4": a power of two, UE8M0) [pages, block_size, heads, head_dim / G].
A batch is block_table [seqs, max_blocks], seq_lens [seqs] (the tokens in the cache, the call's own rows included) and
row_start [seqs + 1]: rows row_start[s] .. row_start[s + 1] are the last tokens of sequence s."""
import math

import torch

own = False

GROUP = {"nvfp4": 16, "mxfp4": 32}
TSCALE = 1.0 / 64.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # The queries of a decode batch: slices of the merged projection's rows.
        {"name": "rope_8x40x128", "op": "rope", "rows": 8, "heads": 40, "head_dim": 128, "rot": 128,
         "interleaved": False, "type": "bf16", "far": 8192},
        # The queries of a long prefill, half of each head rotated, positions beyond the length trained on.
        {"name": "rope_8192x40x128", "op": "rope", "rows": 8192, "heads": 40, "head_dim": 128, "rot": 64,
         "interleaved": True, "type": "f16", "far": 1 << 20},
        # One token of each of 32 streams into the cache.
        {"name": "append_32x1", "op": "append", "fmt": "nvfp4", "type": "bf16", "seqs": 32, "rows": 32, "context": 4096,
         "heads": 8, "head_dim": 128, "block": 16, "rot": 128, "interleaved": False},
        # A prefill chunk of one sequence.
        {"name": "append_1x2048", "op": "append", "fmt": "nvfp4", "type": "bf16", "seqs": 1, "rows": 2048,
         "context": 8192, "heads": 8, "head_dim": 128, "block": 16, "rot": 128, "interleaved": False},
        # A batch of prompts of different lengths into the other format.
        {"name": "append_7x16384", "op": "append", "fmt": "mxfp4", "type": "f16", "seqs": 7, "rows": 16384,
         "context": 0, "heads": 8, "head_dim": 128, "block": 24, "rot": 64, "interleaved": True},
        # One user's decode step early in a conversation: latency counts.
        {"name": "attend_1x1of1000", "op": "attend", "fmt": "nvfp4", "type": "bf16", "seqs": 1, "rows": 1,
         "context": 999, "ragged": False, "heads": 8, "group": 5, "head_dim": 128, "block": 16, "window": 0,
         "padded": 0, "mixed": False},
        # A decode step of 16 streams whose contexts go from 1024 to 8192 tokens.
        {"name": "attend_16x1of8192", "op": "attend", "fmt": "nvfp4", "type": "bf16", "seqs": 16, "rows": 16,
         "context": 8191, "ragged": True, "heads": 8, "group": 5, "head_dim": 128, "block": 16, "window": 0,
         "padded": 0, "mixed": False},
        # One long document.
        {"name": "attend_1x1of131072", "op": "attend", "fmt": "mxfp4", "type": "f16", "seqs": 1, "rows": 1,
         "context": 131071, "ragged": False, "heads": 8, "group": 5, "head_dim": 128, "block": 64, "window": 0,
         "padded": 0, "mixed": False},
        # Four drafted tokens of each of 8 streams verified at once, in a layer that looks 4096 tokens back.
        {"name": "attend_8x4of16384", "op": "attend", "fmt": "nvfp4", "type": "bf16", "seqs": 8, "rows": 32,
         "context": 16380, "ragged": True, "heads": 4, "group": 8, "head_dim": 128, "block": 16, "window": 4096,
         "padded": 0, "mixed": False},
        # A prefill chunk behind 6144 tokens.
        {"name": "attend_1x2048of8192", "op": "attend", "fmt": "nvfp4", "type": "bf16", "seqs": 1, "rows": 2048,
         "context": 6144, "ragged": False, "heads": 8, "group": 5, "head_dim": 128, "block": 16, "window": 0,
         "padded": 0, "mixed": False},
        # Prompts of different lengths, small heads, pages that end inside any power of two.
        {"name": "attend_7x1023", "op": "attend", "fmt": "mxfp4", "type": "f16", "seqs": 7, "rows": 7161,
         "context": 0, "ragged": True, "heads": 4, "group": 4, "head_dim": 64, "block": 24, "window": 0, "padded": 0,
         "mixed": False},
        # A prompt's chunk together with other streams' single tokens, the batch padded to a captured size.
        {"name": "attend_9x264of2303", "op": "attend", "fmt": "nvfp4", "type": "f16", "seqs": 9, "rows": 264,
         "context": 2047, "ragged": True, "heads": 2, "group": 8, "head_dim": 256, "block": 32, "window": 0,
         "padded": 24, "mixed": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    head_dim = rng.choice([64, 96, 128, 128, 256])
    rot = rng.choice([head_dim, head_dim // 2])
    if op == "rope":
        heads = _log(rng, 1, 64)
        return {"op": op, "rows": _log(rng, 1, min(8192, 8192 * 5120 // (heads * head_dim))), "heads": heads,
                "head_dim": head_dim, "rot": rot, "interleaved": rng.random() < 0.5,
                "type": rng.choice(["bf16", "f16"]), "far": _log(rng, 1024, 1 << 20)}
    heads, block = rng.choice([1, 2, 4, 8, 8, 10]), rng.choice([16, 24, 64, 128])
    case = {"op": op, "fmt": rng.choice(["nvfp4", "mxfp4"]), "type": rng.choice(["bf16", "f16"]),
            "seqs": _log(rng, 1, 64), "heads": heads, "head_dim": head_dim, "block": block}
    if op == "append":
        seqs = case["seqs"]
        rows = rng.choice([seqs, max(seqs, _log(rng, 1, min(16384, 16384 * 1024 // (heads * head_dim))))])
        return {**case, "rows": rows, "context": _log(rng, 16, 16384), "rot": rng.choice([rot, 0]),
                "interleaved": rng.random() < 0.5}
    case.update(group=rng.choice([1, 4, 5, 8]), ragged=rng.random() < 0.7, window=rng.choice([0, 0, 1024]),
                padded=rng.choice([0, 0, 5]), mixed=False)
    if rng.random() < 0.6:  # a few rows of each sequence
        per, longest = rng.choice([1, 1, 2, 5]), min(65536, 262144 // case["seqs"])
        return {**case, "rows": per * case["seqs"], "context": _log(rng, 16, longest * 128 // (per * head_dim))}
    # Chunks, alone or among single tokens; all rows times all tokens bounded as in the listed ones.
    seqs = case["seqs"] = min(case["seqs"], 8)
    rows = max(seqs, _log(rng, 64, 2048))
    tokens = max(16, min(8192, 2 ** 29 // (seqs * heads * case["group"] * rows) - rows))
    return {**case, "rows": rows, "context": _log(rng, 16, tokens), "mixed": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _split(total, parts, gen, even):
    """`total` rows over `parts` sequences, at least one each (in equal parts, or uniformly at random)."""
    if even or parts == 1:
        n = torch.full((parts,), total // parts, device="cuda")
        n[:total % parts] += 1
        return n
    cut = torch.rand((parts,), generator=gen, device="cuda").cumsum(0)
    edge = (cut / cut[-1] * (total - parts)).round().long() + torch.arange(1, parts + 1, device="cuda")
    return torch.diff(edge, prepend=edge.new_zeros(1))


def _rotation(rot, gen):
    """Angular frequencies of a long-context model, in radians a token: the slow half slowed eight times more."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    freqs = 1e6 ** (-2 * i / rot)
    slow = ((i - rot / 8) / (rot / 8)).clamp(0, 1)
    return freqs * (1 - slow + slow / 8)


def _channels(heads, head_dim, gen):
    """Keys have a few channels that are several times as large as the rest."""
    return 1 + 3 * (torch.rand((heads, head_dim), generator=gen, device="cuda") < 0.03).float()


def _pages(fmt, pages, block, heads, head_dim, spread, gen):
    """Pages of old tokens: codes and scales of normal values times `spread` [heads, head_dim]."""
    g = GROUP[fmt]
    codes = torch.empty((pages, block, heads, head_dim // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, block, heads, head_dim // g), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (block * heads * head_dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        v = (_normal((n, block, heads, head_dim), gen) * spread).unflatten(-1, (-1, g))
        c, s = _encode(fmt, v, torch.tensor(TSCALE, device="cuda"))
        codes[p:p + n], scales[p:p + n] = c, s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    dt = TYPES[case["type"]]
    if case["op"] == "rope":
        rows, heads, d = case["rows"], case["heads"], case["head_dim"]
        merged = _normal((rows, (heads + 2) * d), gen).to(dt)  # queries, a key and a value head
        s["x"] = merged[:, :heads * d].unflatten(1, (heads, d))
        s["positions"] = torch.randint(0, case["far"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
        s["freqs"], s["amplitude"] = _rotation(case["rot"], gen), 1.1
        return s
    seqs, rows, heads, d, block = case["seqs"], case["rows"], case["heads"], case["head_dim"], case["block"]
    append = case["op"] == "append"
    even = rows == seqs if append else not case["ragged"] or rows == seqs or case["context"] >= 8 * (rows // seqs)
    n = _split(rows, seqs, gen, even)
    if not append and case["mixed"]:  # one sequence's chunk among single tokens
        n = torch.ones_like(n)
        n[seqs // 2] = rows - seqs + 1
    past = torch.full_like(n, case["context"])
    if not append and case["ragged"] and case["context"]:
        past = (case["context"] * (0.125 + 0.875 * torch.rand((seqs,), generator=gen, device="cuda"))).long()
    lens = past + n
    pages = (lens + block - 1) // block
    most, total = (case["context"] + rows + block - 1) // block, int(pages.sum())
    order = torch.randperm(total + 8, generator=gen, device="cuda")[:total].to(torch.int32)
    table = torch.full((seqs, most), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(most, device="cuda") < pages[:, None]] = order
    s["block_table"], s["seq_lens"] = table, lens.to(torch.int32)
    s["row_start"] = None if rows == seqs and not case.get("padded") \
        else torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    channels = _channels(heads, d, gen)
    s["k_codes"], s["k_scales"] = _pages(case["fmt"], total + 8, block, heads, d, channels, gen)
    s["v_codes"], s["v_scales"] = _pages(case["fmt"], total + 8, block, heads, d, 0.5, gen)
    s["k_tscale"], s["v_tscale"] = (torch.full((1,), TSCALE, device="cuda") if case["fmt"] == "nvfp4" else None
                                    for _ in range(2))
    if append:
        merged = _normal((rows, 2 * heads * d), gen)  # keys and values of the merged projection
        merged[:, :heads * d] *= channels.flatten()
        merged = merged.to(dt)
        s["k"], s["v"] = (merged[:, i * heads * d:(i + 1) * heads * d].unflatten(1, (heads, d)) for i in range(2))
        s["freqs"], s["amplitude"] = (_rotation(case["rot"], gen), 1.0) if case["rot"] else (None, 1.0)
        return s
    s["q"] = _normal((rows + case["padded"], heads * case["group"], d), gen, 2.0).to(dt)
    s["out"] = torch.zeros_like(s["q"]) if case["padded"] else None
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    if s["op"] == "rope":
        return _rotate(s["x"].float(), s["positions"], s["freqs"], s["amplitude"], s["interleaved"]).to(s["x"].dtype)
    return _append(s) if s["op"] == "append" else _attend(s)


def _own(s):
    import nvfp4_weight_only_amd as nv
    # A program builds the handles of its rotation and of a layer's cache once and keeps them.
    if "rope" not in s:
        s["rope"] = nv.Rope(s["freqs"], amplitude=s["amplitude"], interleaved=s["interleaved"]) \
            if s.get("freqs") is not None else None
    if s["op"] == "rope":
        return nv.rope(s["x"], s["positions"], s["rope"])
    if "cache" not in s:
        s["cache"] = nv.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], k_tscale=s["k_tscale"],
                                v_tscale=s["v_tscale"], fmt=s["fmt"])
    if s["op"] == "append":
        nv.kv_append(s["k"], s["v"], s["cache"], s["block_table"], s["seq_lens"], row_start=s["row_start"],
                     rope=s["rope"])
        return _cache(s)
    return nv.kv_attention(s["q"], s["cache"], s["block_table"], s["seq_lens"], row_start=s["row_start"],
                           window=s["window"] or None, out=s["out"])


def _cache(s):
    """The cache: scales as the values they stand for; a byte of codes is two values, and equal bytes are asked."""
    view = torch.float8_e4m3fn if s["fmt"] == "nvfp4" else torch.float8_e8m0fnu
    return s["k_codes"], s["k_scales"].view(view), s["v_codes"], s["v_scales"].view(view)


def _rotate(x, positions, freqs, amplitude, interleaved):
    """x [rows, heads, head_dim] in 32 or 64 bits; angles in 64 bits."""
    angle = positions.double()[:, None] * freqs
    cos, sin = ((f(angle) * amplitude).to(x.dtype)[:, None] for f in (torch.cos, torch.sin))
    rot = 2 * freqs.numel()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = [a * cos - b * sin, b * cos + a * sin]
    return torch.cat([torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1), x[..., rot:]], -1)


def _nearest(x, mids):
    """The number of the grid value nearest to x, of neighbours with equal distance the even one."""
    below, upto = torch.bucketize(x, mids, out_int32=True), torch.bucketize(x, mids, out_int32=True, right=True)
    return torch.where(below % 2 == 0, below, upto)


def _e4m3_grid(device):
    return torch.arange(127, device=device, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def _encode(fmt, v, tscale):
    """v [..., blocks, G] in 32 bits -> codes [..., blocks * G / 2], scales [..., blocks]; quotients in 64 bits, since
    a value next to a border decides by its last bits."""
    amax = v.abs().amax(-1)
    if fmt == "nvfp4":
        grid = _e4m3_grid(v.device)
        scale = _nearest(amax.double() / (6 * tscale.double()), (grid[1:] + grid[:-1]) / 2)
        unit = (grid[scale.long()] * tscale.double())[..., None]
    else:
        scale = (torch.frexp(amax).exponent - 3 + 127).clamp(0, 254)
        scale = torch.where(amax > 0, scale, 0)
        unit = torch.exp2(scale.double() - 127)[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=v.device)
    code = _nearest(torch.where(unit > 0, v.abs().double() / unit, 0.0), mids).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., ::2] | code[..., 1::2] << 4, scale.to(torch.uint8)


def _append(s):
    rows, fmt, table = s["rows"], s["fmt"], s["block_table"].long()
    row, lens = torch.arange(rows, device=table.device), s["seq_lens"].long()
    start = torch.arange(len(lens) + 1, device=table.device) if s["row_start"] is None else s["row_start"].long()
    seq = torch.bucketize(row, start[1:], right=True)
    pos = lens[seq] - (start[seq + 1] - row)
    page, slot = table[seq, pos // s["block"]], pos % s["block"]
    k, v = s["k"].float(), s["v"].float()
    if s["freqs"] is not None:  # in 64 bits and rounded once, since the codes hang on borders
        k = _rotate(s["k"].double(), pos, s["freqs"], s["amplitude"], s["interleaved"]).float()
    for name, x in (("k", k), ("v", v)):
        codes, scales = _encode(fmt, x.unflatten(-1, (-1, GROUP[fmt])), s[name + "_tscale"])
        s[name + "_codes"][page, slot], s[name + "_scales"][page, slot] = codes, scales
    return _cache(s)


def _decode(s, name, page, slot):
    """The tokens at (page, slot) in 32 bits: [..., heads, head_dim]."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=page.device)
    pairs = torch.stack([e2m1.repeat(16), e2m1.repeat_interleave(16)], -1)  # by byte: low nibble, high nibble
    x = pairs[s[name + "_codes"][page, slot].int()].flatten(-2).unflatten(-1, (-1, GROUP[s["fmt"]]))
    scale = s[name + "_scales"][page, slot]
    if s["fmt"] == "nvfp4":
        scale = scale.view(torch.float8_e4m3fn).float() * s[name + "_tscale"]
    else:
        scale = scale.view(torch.float8_e8m0fnu).float()
    return (x * scale[..., None]).flatten(-2)


def _attend(s):
    q, table, lens = s["q"], s["block_table"].long(), s["seq_lens"].long()
    seqs, rows, d = len(lens), s["rows"], s["head_dim"]
    start = torch.arange(seqs + 1, device=q.device) if s["row_start"] is None else s["row_start"].long()
    # Every sequence padded to the longest one's tokens and rows.
    tokens = torch.arange(int(lens.max()), device=q.device)
    count = start.diff()
    page = table[:, tokens // s["block"]].clamp(min=0)
    # [seqs, heads, tokens, d], and queries [seqs, heads, group * rows, d]
    k, v = (_decode(s, n, page, tokens % s["block"]).permute(0, 2, 1, 3) for n in ("k", "v"))
    i = torch.arange(int(count.max()), device=q.device)
    row = (start[:-1, None] + i).clamp(max=rows - 1)
    pos = (lens - count)[:, None] + i                              # of row i of each sequence
    x = q[row].float().unflatten(2, (s["heads"], -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (x @ k.transpose(2, 3)).mul_(d ** -0.5).unflatten(2, (-1, len(i)))
    seen = tokens <= pos[..., None]
    if s["window"]:
        seen &= tokens > pos[..., None] - s["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)            # a row that sees nothing: exp(-inf) = 0
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    y = (score.flatten(2, 3) @ v).unflatten(2, (-1, len(i))) / total.clamp(min=1e-38)
    y = y.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)         # [seqs, rows, q heads, d]
    out = torch.empty_like(q) if s["out"] is None else s["out"]
    mine = i < count[:, None]
    out[row[mine]] = y[mine]
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    d, rows = case["head_dim"], case["rows"]
    if case["op"] == "rope":
        return {"bytes": 4 * rows * case["heads"] * d + 4 * rows + 4 * case["rot"],
                "flops": 3 * rows * case["heads"] * case["rot"]}
    heads, seqs = case["heads"], case["seqs"]
    token = 2 * heads * (d // 2 + d // GROUP[case["fmt"]])  # a token's keys and values in the cache
    if case["op"] == "append":
        return {"bytes": 4 * rows * heads * d + rows * token, "flops": rows * heads * (3 * case["rot"] + 6 * d)}
    # Contexts of ragged batches are 9/16 of the longest on average; rows see a triangle of their own tokens.
    past = case["context"] * (9 / 16 if case["ragged"] and case["context"] else 1)
    chunks = [1] * (seqs - 1) + [rows - seqs + 1] if case["mixed"] else [rows / seqs] * seqs
    tokens = pairs = 0
    for n in chunks:
        seen = past + (n + 1) / 2
        if case["window"]:
            seen = min(seen, case["window"])
        pairs += n * seen
        tokens += min(past + n, case["window"] + n) if case["window"] else past + n
    q_heads = heads * case["group"]
    return {"bytes": tokens * token + 4 * rows * q_heads * d, "flops": 4 * pairs * q_heads * d}


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _turn(x, pos, freqs, amplitude, interleaved):
    """Pairs as complex numbers times amplitude * e^(i * position * frequency)."""
    half = freqs.numel()
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.full_like(freqs, amplitude), pos.double()[:, None] * freqs)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _values(s, name, page, slot):
    """Tokens of the cache in 64 bits, from the formats' fields."""
    byte = s[name + "_codes"][page, slot].long()
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    exp, man = (code >> 1) & 3, (code & 1).double()
    x = torch.where(exp > 0, (1 + man / 2) * torch.exp2(exp.double() - 1), man / 2) * (1 - 2 * (code >> 3)).double()
    b = s[name + "_scales"][page, slot].long()
    if s["fmt"] == "nvfp4":
        exp, man = b >> 3, (b & 7).double()
        scale = torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp.double() - 7), man / 512)
        scale = scale * s[name + "_tscale"].double()
    else:
        scale = torch.exp2(b.double() - 127)
    return x * scale.repeat_interleave(GROUP[s["fmt"]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _turn(s["x"].double(), s["positions"], s["freqs"], s["amplitude"], s["interleaved"])
    lens, rows = s["seq_lens"].tolist(), s["rows"]
    start = list(range(len(lens) + 1)) if s["row_start"] is None else s["row_start"].tolist()
    table, block = s["block_table"].long(), s["block"]
    if s["op"] == "append":
        return _exact_append(s, lens, start, table)
    q, out = s["q"].double(), torch.zeros_like(s["q"], dtype=torch.float64)
    group, root = case["group"], math.sqrt(case["head_dim"])
    for i, n in enumerate(lens):
        t = torch.arange(n, device=q.device)
        page, slot = table[i, t // block], t % block
        k, v = _values(s, "k", page, slot), _values(s, "v", page, slot)
        r = torch.arange(start[i], start[i + 1], device=q.device)
        pos = n - start[i + 1] + r
        hidden = t > pos[:, None]
        if case["window"]:
            hidden |= t <= pos[:, None] - case["window"]
        for h in range(q.shape[1]):
            score = (q[r, h] @ k[:, h // group].T / root).masked_fill(hidden, -math.inf)
            out[r, h] = torch.softmax(score, -1) @ v[:, h // group]
    return out


def _exact_append(s, lens, start, table):
    """The scales, as values; the codes are whole numbers, which the plain form decides in 64 bits too."""
    found = []
    for name in ("k", "v"):
        x, fmt = s[name].double(), s["fmt"]
        cache = s[name + "_scales"]
        scales = cache.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(cache.double() - 127)
        for i, n in enumerate(lens):
            r = torch.arange(start[i], start[i + 1], device=x.device)
            t = n - start[i + 1] + r
            y = _turn(x[r], t, s["freqs"], s["amplitude"], s["interleaved"]) if name == "k" and s["rot"] else x[r]
            top = y.unflatten(-1, (-1, GROUP[fmt])).abs().amax(-1)
            if fmt == "nvfp4":
                # Below 2^-6 E4M3's step is 2^-9, above it an eighth of the power of two; round() takes ties to even.
                want = (top / 6 / s[name + "_tscale"].double()).clamp(max=448)
                step = torch.exp2(torch.frexp(want.clamp(min=2.0 ** -6)).exponent.double() - 4)
                unit = (want / step).round() * step
            else:
                unit = torch.exp2(torch.floor(torch.log2(top)) - 2).clamp(min=2.0 ** -127)
            scales[table[i, t // s["block"]], t % s["block"]] = unit
        found += [None, scales]
    return tuple(found)
