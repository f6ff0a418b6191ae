"""CPU oracle for the operators around a paged FP4 cache: rotary positions, appending, attention.  TEST INFRASTRUCTURE
ONLY: it shares no code, table or helper with the HIP path.

Plain numpy in float64.  Formats, tables and decoding are those of nvfp4_oracle and kv_oracle (R14, R15; here without
the rounding to 16 bits).

  R25 rotation   pairs (i, i + rot / 2), or interleaved (2 i, 2 i + 1), of the first rot elements of a head turned by
                 t = position * freqs[i]: amplitude * (x1 cos t - x2 sin t, x2 cos t + x1 sin t).
  R26 placement  rows row_start[s] .. row_start[s + 1] - 1 are the last tokens of sequence s: row r is token
                 seq_lens[s] - (row_start[s + 1] - r), in page block_table[s, t // block_size]; rows of no sequence,
                 tokens below 0 or past the table and pages outside [0, num_blocks) are skipped.
  R27 encoding   NVFP4 with the cache's tensor scale: E4M3 nearest to amax / (6 tscale), at most 448; E2M1 nearest to
                 |x| / (scale tscale), at most 6; ties to the even code.  MXFP4: R17.  Values that are not finite: NaN
                 scale, codes 0.  A turned key is rounded to float32 first.
  R28 attention  softmax(scale q . k_t) over the tokens t <= p, t > p - window, that are in the cache; a row that sees
                 nothing gives zeros.  MXFP4 blocks whose byte is 253 or 254 count as NaN, like 255.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.kv_oracle import GROUP, MXFP4, NVFP4, UE8M0_TABLE
from oracle.nvfp4_oracle import (E2M1_TABLE, E4M3_TABLE, _E2M1_MIDS, _E4M3_MIDS, _nearest_code_ties_even, pack_nibbles,
                                 unpack_nibbles)


def rotate(x, positions, freqs, amplitude=1.0, interleaved=False):
    """R25: x [rows, heads, head_dim] float64."""
    x = np.array(x, dtype=np.float64)
    half = len(freqs)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    cos, sin = np.cos(angle)[:, None] * amplitude, np.sin(angle)[:, None] * amplitude
    first = np.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    a, b = x[..., first], x[..., second]
    x[..., first], x[..., second] = a * cos - b * sin, b * cos + a * sin
    return x


def frequencies(scaling, rot, base, factor=1.0, original=0.0, low=1.0, high=32.0):
    """float64 [rot / 2], from the formulas in plain Python floats."""
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling in ("ramp", "wavelength"):
            if scaling == "ramp":
                def at(n):
                    return rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
                a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
                w = (i - a) / max(b - a, 0.001)
            else:
                w = (high - original * f / (2 * math.pi)) / (high - low)
            w = min(max(w, 0.0), 1.0)
            f = f * (1 - w) + f / factor * w
        out.append(f)
    return np.array(out)


def encode(fmt, x, tscale=None):
    """R27: x [..., D] float64 (float32 values) -> (codes [..., D/2], scales [..., D/G])."""
    g = GROUP[fmt]
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, g)
    bad = ~np.isfinite(blocks).all(-1)
    v = np.where(bad[..., None], 0.0, blocks)
    amax = np.abs(v).max(-1)
    if fmt == NVFP4:
        ts = np.float64(np.float32(tscale))
        scale = _nearest_code_ties_even(amax, _E4M3_MIDS, 6 * ts * np.ones_like(amax)).astype(np.uint8)
        scale[amax == 0] = 0
        unit = (E4M3_TABLE[scale] * ts)[..., None]
        code = _nearest_code_ties_even(np.abs(v), _E2M1_MIDS, unit)
        code[np.broadcast_to(unit == 0, code.shape)] = 0
        scale[bad] = 0x7F
    else:
        e = np.zeros(amax.shape, dtype=np.int64)
        nz = amax > 0
        _, ex = np.frexp(amax[nz])
        e[nz] = np.clip(ex.astype(np.int64) - 3 + 127, 0, 254)
        scale = e.astype(np.uint8)
        code = _nearest_code_ties_even(np.abs(v), _E2M1_MIDS, np.ldexp(1.0, e - 127)[..., None])
        scale[bad] = 0xFF
    code = (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)
    code[bad] = 0
    return pack_nibbles(code.reshape(-1, x.shape[-1])).reshape(*x.shape[:-1], -1), scale


def values(fmt, codes, scales, tscale=None):
    """E2M1 * scale (* tscale) in float64."""
    g = GROUP[fmt]
    e2m1 = E2M1_TABLE[unpack_nibbles(codes.reshape(-1, codes.shape[-1]))].reshape(*codes.shape[:-1], -1)
    sc = np.repeat((E4M3_TABLE if fmt == NVFP4 else UE8M0_TABLE)[scales], g, axis=-1)
    with np.errstate(invalid="ignore"):
        return e2m1 * sc * (np.float64(np.float32(tscale)) if fmt == NVFP4 else 1.0)


def places(rows, block_table, seq_lens, row_start, num_blocks, block_size):
    """R26: for each row (sequence, token, page, slot), page -1 where it is skipped, sequence -1 where it has none."""
    seqs, max_blocks = block_table.shape
    out = [(-1, -1, -1, -1)] * rows
    for s in range(seqs):
        a, e = (s, s + 1) if row_start is None else (int(row_start[s]), int(row_start[s + 1]))
        for r in range(max(a, 0), min(e, rows)):
            t = int(seq_lens[s]) - (e - r)
            page = -1
            if 0 <= t < max_blocks * block_size:
                page = int(block_table[s, t // block_size])
                page = page if 0 <= page < num_blocks else -1
            out[r] = (s, t, page, t % block_size)
    return out


def append(fmt, cache, k, v, block_table, seq_lens, row_start=None, freqs=None, amplitude=1.0, interleaved=False,
           positions=None):
    """R26, R27: cache = {"k_codes", "k_scales", "k_tscale", "v_..."} (uint8 arrays) -> the same after the call."""
    cache = {n: (c.copy() if isinstance(c, np.ndarray) else c) for n, c in cache.items()}
    nb, bs = cache["k_codes"].shape[:2]
    at = places(len(k), block_table, seq_lens, row_start, nb, bs)
    with np.errstate(invalid="ignore", over="ignore"):
        if freqs is not None:
            pos = [p[1] for p in at] if positions is None else positions
            k = rotate(k, pos, freqs, amplitude, interleaved).astype(np.float32)
    for name, x in (("k", k), ("v", v)):
        codes, scales = encode(fmt, x, cache[name + "_tscale"])
        for r, (_, _, page, slot) in enumerate(at):
            if page >= 0:
                cache[name + "_codes"][page, slot], cache[name + "_scales"][page, slot] = codes[r], scales[r]
    return cache


def attention(fmt, cache, q, block_table, seq_lens, row_start, scale, window, weight_step):
    """R28: (y, bound, mine): float64 outputs, how far a kernel's may be off before the output's rounding, and the rows
    that belong to a sequence.

    The bound, with u = 2^-24 (half a step of FP32), A_t = |scale| sum |q_i k_ti|: the products' FP32 sum over D elements
    and the scaling are off by (D + 4) u A_t, elements of q below its row's maximum by 2^-25 of it, the difference from
    the maximum and its base change by 4 u |s_t|, exp2 by 2^-22; a weight's relative error is e to that, so twice the
    exponent's error, plus its rounding (weight_step); sums over n tokens and the joins n u.  Each moves the output by
    sum w |v| / sum w at most, numerator and denominator alike.  Weights in FP16 that lie more than 2^21 below the largest,
    whose own is at least 2^7 there, are its subnormals: off by 2^-25 / 2^7 of the largest, 2^-32 sum |v| / sum w.  With
    MXFP4 a row's largest weight is held as 2^-8 to 1 (so that sums of its largest values stay in FP32's range), and what
    falls below FP32's smallest normal number, 2^-126, may be 0: 2^-126 / 2^-8 of the largest, 2^-118 sum |v| / sum w."""
    nb, bs, heads, half = cache["k_codes"].shape
    rows, q_heads, d = q.shape
    y, bound, mine = np.zeros((rows, q_heads, d)), np.zeros((rows, q_heads, d)), np.zeros(rows, dtype=bool)
    u = 2.0 ** -24
    kv = [values(fmt, cache[n + "_codes"],
                 np.where(cache[n + "_scales"] >= 253, 255, cache[n + "_scales"]) if fmt == MXFP4 else cache[n + "_scales"],
                 cache[n + "_tscale"]) for n in "kv"]
    for r, (s, p, _, _) in enumerate(places(rows, block_table, seq_lens, row_start, nb, bs)):
        if s < 0:
            continue
        mine[r] = True
        lo = max(0, p - window + 1) if window else 0
        t = np.arange(lo, min(p + 1, int(seq_lens[s]), block_table.shape[1] * bs))
        page = block_table[s, t // bs]
        ok = (page >= 0) & (page < nb)
        page, slot = page[ok], (t % bs)[ok]
        if len(page) == 0:
            continue
        k, v = (np.repeat(x[page, slot], q_heads // heads, axis=1) for x in kv)  # [n, q_heads, d]
        with np.errstate(invalid="ignore", over="ignore"):
            sc = scale * np.einsum("hd,nhd->nh", q[r], k)
            size = abs(scale) * np.einsum("hd,nhd->nh", np.abs(q[r]), np.abs(k))
            top = sc.max(0)
            w = np.exp(sc - top)
            total = w.sum(0)[:, None]
            y[r] = np.einsum("nh,nhd->hd", w, v) / total
            spread = np.einsum("nh,nhd->hd", w, np.abs(v)) / total
            qmax = np.abs(q[r]).max(-1)
            far = (d + 4) * u * size + 4 * u * np.abs(sc) + 4 * u * np.abs(top) \
                + 2.0 ** -25 * qmax * abs(scale) * np.abs(k).sum(-1)
            bound[r] = spread * (4 * far.max(0) + 2 * weight_step + 2.0 ** -21 + 2 * (len(page) + 16) * u)[:, None]
            bound[r] += (2.0 ** -32 if fmt == NVFP4 else 2.0 ** -118) * np.abs(v).sum(0) / total
    return y, bound, mine
