"""The operators around a paged FP4 cache (rotary positions, appending, attention): refusals of the C entry points and
the binding (CPU), and the HIP kernels against the float64 oracle (GPU)."""
import ctypes
import itertools
import os

import numpy as np
import pytest
import torch

from nvfp4_weight_only_amd import binding as B
from nvfp4_weight_only_amd import build as BUILD
from oracle import kv_ops_oracle as K
from oracle import mxfp4_oracle as MX
from oracle import nvfp4_oracle as O

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest subnormal
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.lib_path()):
        BUILD.build()
    return B.lib()


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_weight_only_amd as nv
    nv.lib()
    return nv


# ---------------------------------------------------------------------------
# CPU: the oracle, and what the entry points refuse.
# ---------------------------------------------------------------------------
def test_oracle_encode_matches_the_quantizers():
    rng = np.random.default_rng(0)
    w = O.f32_to_bf16_rne(rng.normal(size=(6, 64)).astype(np.float32))
    x = O.bf16_to_f64(w)
    codes, scales = K.encode("mxfp4", x)
    pm, sm = MX.quantize(w)
    assert np.array_equal(codes, pm) and np.array_equal(scales, sm)
    # With amax = 2688 tscale exactly, the cache's rule is the weights' rule.
    w[0, 0] = O.f32_to_bf16_rne(np.array([8.0], np.float32))[0]
    codes, scales = K.encode("nvfp4", O.bf16_to_f64(w), 8.0 / 2688)
    pn, sn, ts = O.quantize(w)
    assert np.array_equal(scales, sn) and (codes == pn).mean() > 0.999


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x, pos, freqs = rng.normal(size=(3, 2, 48)), [0, 7, -5], K.frequencies(None, 32, 1e4)
    for il in (False, True):
        y = K.rotate(x, pos, freqs, interleaved=il)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose(K.rotate(y, [0, -7, 5], freqs, interleaved=il), x)


# Fake, never-dereferenced device addresses: validation fails before any HIP call.
A = [i * 0x100000000 for i in range(1, 16)]
BIG = 2 ** 62


def rope_spec(freqs=A[9], rot=64, amplitude=1.0, interleaved=0):
    return B._RopeStruct(freqs, rot, amplitude, interleaved)


def cache_struct(fmt=0, nb=8, bs=16, heads=2, d=64, kc=A[0], ks=A[1], kt=A[2], vc=A[3], vs=A[4], vt=A[5]):
    return B._KvCacheStruct(fmt, nb, bs, heads, d, kc, ks, kt, vc, vs, vt)


def test_rope_validation(L):
    def f(type=1, x=A[0], rows=4, heads=2, d=64, xs=(128, 64), pos=A[1], rope=rope_spec(), inv=0, out=A[2],
          os_=(128, 64)):
        return L.nvfp4_rope(type, x, rows, heads, d, *xs, pos, None if rope is None else ctypes.addressof(rope), inv, out,
                            *os_, None)
    assert f(type=2) == B.ERR_UNSUPPORTED and f(type=-1) == B.ERR_UNSUPPORTED
    assert f(rows=-1) == B.ERR_SHAPE and f(heads=0) == B.ERR_SHAPE and f(d=0) == B.ERR_SHAPE and f(d=68) == B.ERR_SHAPE
    assert f(rope=None) == B.ERR_NULL and f(rope=rope_spec(freqs=None)) == B.ERR_NULL
    for rot in (0, -16, 24, 80):
        assert f(rope=rope_spec(rot=rot)) == B.ERR_SHAPE
    for amp in (float("nan"), float("inf")):
        assert f(rope=rope_spec(amplitude=amp)) == B.ERR_UNSUPPORTED
    assert f(rope=rope_spec(freqs=A[9] + 4)) == B.ERR_ALIGN
    assert f(d=4096, xs=(8192, 4096), os_=(8192, 4096)) == B.ERR_UNSUPPORTED
    assert f(rows=2 ** 31) == B.ERR_UNSUPPORTED
    assert f(xs=(-128, 64)) == B.ERR_SHAPE and f(xs=(128, BIG)) == B.ERR_SHAPE and f(rows=2 ** 30, xs=(BIG, 64)) == B.ERR_SHAPE
    assert f(os_=(120, 64)) == B.ERR_SHAPE and f(os_=(128, 56)) == B.ERR_SHAPE and f(os_=(0, 64)) == B.ERR_SHAPE
    assert f(x=None, rows=0, pos=None, out=None) == B.OK
    assert f(x=None) == B.ERR_NULL and f(pos=None) == B.ERR_NULL and f(out=None) == B.ERR_NULL
    assert f(x=A[0] + 8) == B.ERR_ALIGN and f(pos=A[1] + 2) == B.ERR_ALIGN and f(xs=(132, 64)) == B.ERR_ALIGN
    assert f(out=A[0], os_=(256, 64)) == B.ERR_ALIAS                     # in place, other strides
    assert f(out=A[0] + 16) == B.ERR_ALIAS and f(out=A[1]) == B.ERR_ALIAS and f(out=A[9]) == B.ERR_ALIAS
    assert f(xs=(0, 64), out=A[0] + 256 - 16) == B.ERR_ALIAS             # a broadcast row's last elements


def test_rope_frequencies_validation(L):
    def f(scaling=0, rot=64, base=1e4, factor=1.0, original=0.0, low=1.0, high=32.0, out=A[0]):
        return L.nvfp4_rope_frequencies(scaling, rot, base, factor, original, low, high, out, None)
    assert f(scaling=5) == B.ERR_UNSUPPORTED and f(scaling=-1) == B.ERR_UNSUPPORTED
    assert f(rot=0) == B.ERR_SHAPE and f(rot=20) == B.ERR_SHAPE and f(rot=4096) == B.ERR_SHAPE
    for base in (1.0, 0.0, -3.0, float("nan"), float("inf")):
        assert f(base=base) == B.ERR_UNSUPPORTED
    for factor in (0.5, float("nan"), float("inf")):
        assert f(scaling=1, factor=factor) == B.ERR_UNSUPPORTED
    for kw in ({"original": 0.0}, {"original": 10.0, "low": 0.0}, {"original": 10.0, "low": 4.0, "high": 4.0},
               {"original": float("inf")}, {"original": 10.0, "high": float("inf")}):
        assert f(scaling=3, factor=2.0, **kw) == B.ERR_UNSUPPORTED and f(scaling=4, factor=2.0, **kw) == B.ERR_UNSUPPORTED
    assert f(out=None) == B.ERR_NULL and f(out=A[0] + 4) == B.ERR_ALIGN


CACHE_FAULTS = [({"fmt": 2}, B.ERR_UNSUPPORTED), ({"fmt": -1}, B.ERR_UNSUPPORTED), ({"nb": 0}, B.ERR_SHAPE),
                ({"bs": -1}, B.ERR_SHAPE), ({"heads": 0}, B.ERR_SHAPE), ({"d": 0}, B.ERR_SHAPE), ({"d": 72}, B.ERR_SHAPE),
                ({"fmt": 1, "d": 80}, B.ERR_SHAPE), ({"nb": BIG}, B.ERR_SHAPE), ({"kc": None}, B.ERR_NULL),
                ({"vs": None}, B.ERR_NULL), ({"kt": None}, B.ERR_NULL), ({"vt": None}, B.ERR_NULL),
                ({"d": 4096}, B.ERR_UNSUPPORTED), ({"heads": 2 ** 20}, B.ERR_UNSUPPORTED),
                ({"kc": A[0] + 8}, B.ERR_ALIGN), ({"vs": A[4] + 4}, B.ERR_ALIGN), ({"vt": A[5] + 2}, B.ERR_ALIGN)]
BATCH_FAULTS = [({"rows": -1}, B.ERR_SHAPE), ({"seqs": -1}, B.ERR_SHAPE), ({"max_blocks": 0}, B.ERR_SHAPE),
                ({"max_blocks": BIG}, B.ERR_SHAPE), ({"start": None}, B.ERR_SHAPE),
                ({"max_blocks": 2 ** 27}, B.ERR_UNSUPPORTED), ({"rows": 2 ** 31}, B.ERR_UNSUPPORTED),
                ({"table": None}, B.ERR_NULL), ({"lens": None}, B.ERR_NULL), ({"table": A[7] + 1}, B.ERR_ALIGN),
                ({"lens": A[8] + 2}, B.ERR_ALIGN), ({"start": A[10] + 2}, B.ERR_ALIGN)]


def append_args(cache=None, type=1, k=A[6], v=A[11], rows=4, ks=(128, 64), vs=(128, 64), table=A[7], max_blocks=4,
                lens=A[8], start=A[10], seqs=2, rope=None, positions=None):
    return (None if cache is None else ctypes.addressof(cache), type, k, v, rows, *ks, *vs, table, max_blocks, lens, start,
            seqs, None if rope is None else ctypes.addressof(rope), positions, None)


def test_kv_append_validation(L):
    good = cache_struct()

    def f(cache=good, **kw):
        return L.nvfp4_kv_append(*append_args(cache, **kw))
    assert f(cache=None) == B.ERR_NULL
    for kw, err in CACHE_FAULTS:
        assert f(cache=cache_struct(**kw)) == err, kw
    for kw, err in BATCH_FAULTS:
        assert f(**kw) == err, kw
    assert f(type=2) == B.ERR_UNSUPPORTED
    assert f(rope=rope_spec(rot=80)) == B.ERR_SHAPE and f(rope=rope_spec(freqs=None)) == B.ERR_NULL
    assert f(rows=0) == B.OK and f(seqs=0) == B.OK and f(rows=0, k=None, v=None, table=None, lens=None) == B.OK
    assert f(k=None) == B.ERR_NULL and f(v=None) == B.ERR_NULL
    assert f(k=A[6] + 8) == B.ERR_ALIGN and f(vs=(132, 64)) == B.ERR_ALIGN
    assert f(rope=rope_spec(), positions=A[12] + 1) == B.ERR_ALIGN
    assert f(ks=(-8, 64)) == B.ERR_SHAPE
    # Outputs over inputs or each other.
    assert f(k=A[0]) == B.ERR_ALIAS and f(v=A[4]) == B.ERR_ALIAS and f(table=A[1]) == B.ERR_ALIAS
    assert f(lens=A[3]) == B.ERR_ALIAS and f(start=A[0] + 16) == B.ERR_ALIAS
    assert f(rope=rope_spec(freqs=A[1])) == B.ERR_ALIAS and f(rope=rope_spec(), positions=A[3]) == B.ERR_ALIAS
    assert f(cache=cache_struct(vc=A[0])) == B.ERR_ALIAS and f(cache=cache_struct(kt=A[4] + 4)) == B.ERR_ALIAS


def test_kv_attention_validation(L):
    need = L.nvfp4_kv_attention_workspace_bytes(2, 64, 4, 4, 2)
    assert need > 0
    good = cache_struct()

    def f(cache=good, type=1, q=A[6], rows=4, q_heads=4, qs=(256, 64), table=A[7], max_blocks=4, lens=A[8], start=A[10],
          seqs=2, scale=0.125, window=0, out=A[11], ws=A[12], wsb=need):
        return L.nvfp4_kv_attention(None if cache is None else ctypes.addressof(cache), type, q, rows, q_heads, *qs, table,
                                    max_blocks, lens, start, seqs, scale, window, out, ws, wsb, None)
    assert f(cache=None) == B.ERR_NULL
    for kw, err in CACHE_FAULTS:
        assert f(cache=cache_struct(**kw)) == err, kw
    for kw, err in BATCH_FAULTS:
        assert f(**kw) == err, kw
    assert f(type=2) == B.ERR_UNSUPPORTED and f(scale=float("nan")) == B.ERR_UNSUPPORTED
    assert f(scale=float("inf")) == B.ERR_UNSUPPORTED
    assert f(q_heads=0) == B.ERR_SHAPE and f(q_heads=3) == B.ERR_SHAPE and f(window=-1) == B.ERR_SHAPE
    assert f(wsb=-1) == B.ERR_SHAPE and f(wsb=need - 1) == B.ERR_SHAPE
    for d in (16, 32, 80, 112, 160, 512):
        assert f(cache=cache_struct(d=d), wsb=2 ** 40) == B.ERR_UNSUPPORTED
    assert f(rows=2 ** 29, wsb=2 ** 50) == B.ERR_UNSUPPORTED
    assert f(rows=0, q=None, out=None, ws=None, wsb=0) == B.OK and f(seqs=0, ws=None, wsb=0) == B.OK
    assert f(q=None) == B.ERR_NULL and f(out=None) == B.ERR_NULL and f(ws=None) == B.ERR_NULL
    assert f(q=A[6] + 8) == B.ERR_ALIGN and f(out=A[11] + 8) == B.ERR_ALIGN and f(ws=A[12] + 8) == B.ERR_ALIGN
    assert f(qs=(252, 64)) == B.ERR_ALIGN
    for at in (A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], A[8], A[10]):
        assert f(out=at) == B.ERR_ALIAS and f(ws=at) == B.ERR_ALIAS, hex(at)
    assert f(out=A[12]) == B.ERR_ALIAS
    wb = L.nvfp4_kv_attention_workspace_bytes
    for bad in ((0, 64, 4, 4, 2), (2, 64, 3, 4, 2), (2, 80, 4, 4, 2), (2, 64, 4, -1, 2), (2, 64, 4, 4, -1),
                (2, 64, 4, BIG, 2), (2, 64, BIG, 1, 1)):
        assert wb(*bad) == -1, bad
    assert wb(2, 64, 4, 0, 2) == 0


# ---------------------------------------------------------------------------
# GPU.
# ---------------------------------------------------------------------------
def f64(t):
    return t.detach().double().cpu().numpy()


def rand(rng, shape, dt, std=1.0):
    return torch.from_numpy(rng.normal(0, std, size=shape).astype(np.float32)).to(dt).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_cache(rng, fmt, nb, bs, heads, d, spread=1.0):
    """Random codes, scales around 1/8 .. 8 (times the tensor scale's inverse)."""
    c = {}
    for n in "kv":
        c[n + "_codes"] = rng.integers(0, 256, size=(nb, bs, heads, d // 2), dtype=np.uint8)
        lo, hi = (0x28, 0x48) if fmt == "nvfp4" else (122, 128)
        c[n + "_scales"] = rng.integers(lo, hi + 1, size=(nb, bs, heads, d // K.GROUP[fmt]), dtype=np.uint8)
        c[n + "_tscale"] = np.float32((0.07 if n == "k" else 0.3) * spread) if fmt == "nvfp4" else None
    return c


def device_cache(nv, fmt, c):
    t = {n: None if x is None else torch.from_numpy(np.atleast_1d(x)).cuda() for n, x in c.items()}
    return nv.KVCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], t["k_tscale"], t["v_tscale"], fmt)


def host_cache(cache, c):
    return {**c, **{n: getattr(cache, n).cpu().numpy() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}}


def same_cache(got, want):
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert np.array_equal(got[n], want[n]), f"{n}: {int((got[n] != want[n]).sum())} of {want[n].size} bytes differ"


def make_batch(rng, lens, rows, bs, extra_blocks=1, spare=3):
    """Random distinct pages for sequences of `lens` tokens, the last `rows` of them the call's."""
    pages = [max(0, -(-n // bs)) for n in lens]
    nb = sum(pages) + spare
    order = rng.permutation(nb).astype(np.int32)
    table = np.full((len(lens), max(pages + [1]) + extra_blocks), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    return nb, table, np.array(lens, np.int32), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


ROPE_CASES = [(1, 1, 16, 16, False), (3, 5, 64, 64, True), (7, 40, 128, 128, False), (33, 3, 96, 32, True),
              (5, 2, 80, 48, False), (2, 9, 256, 256, True), (300, 8, 128, 64, False), (1, 1, 2048, 2048, False),
              (9, 1, 24, 16, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "x".join(str(int(v)) for v in c))
def test_rope(nv, case, dt):
    """Against R25.  FP32 sine and cosine (u each), times the amplitude (u), two products and their sum (u each): 4 u
    amplitude (|x1| + |x2|), then half a step of the type."""
    rows, heads, d, rot, il = case
    dt, rng = TYPES[dt], np.random.default_rng(hash(case) % 2 ** 32)
    merged = rand(rng, (rows, heads + 2, d), dt, 2.0)
    x = merged[:, 1:heads + 1]                                   # rows and heads of a merged projection
    pos = rng.integers(-100, 2 ** 20, size=rows)
    freqs = K.frequencies("wavelength", rot, 1e6, 8.0, 4096, 1.0, 4.0)
    r = nv.Rope(torch.from_numpy(freqs).cuda(), amplitude=1.25, interleaved=il)
    for inverse in (False, True):
        want = K.rotate(f64(x), pos, -freqs if inverse else freqs, 1.25, il)
        tol = HALF_STEP[dt] * np.abs(want) + TINY[dt]
        tol[..., :rot] += 4.1 * U * 1.25 * np.sqrt(2) * np.abs(f64(x)).max()
        for out in (None, torch.full_like(merged, 7.0).transpose(0, 1).contiguous().transpose(0, 1)[:, 2:]):
            y = nv.rope(x, i32(pos), r, out=out, inverse=inverse)
            assert (np.abs(f64(y) - want) <= tol).all()
            assert torch.equal(y[..., rot:], x[..., rot:])
    keep = merged.clone()
    y = nv.rope(x, i32(pos), r)
    assert nv.rope(x, i32(pos), r, out=x) is x                   # in place
    assert torch.equal(x, y) and torch.equal(merged[:, 0], keep[:, 0]) and torch.equal(merged[:, -1], keep[:, -1])


@pytest.mark.gpu
def test_rope_gradient(nv):
    """The inverse is the transpose: <rope(x), y> = <x, inverse(y)>, and agrees with differences of a scalar loss."""
    rng = np.random.default_rng(3)
    freqs = K.frequencies(None, 32, 1e4)
    pos = np.array([3, 90000])
    x, y = rng.normal(size=(2, 2, 2, 48))
    for il in (False, True):
        turn = K.rotate(x, pos, freqs, 1.5, il)
        r = nv.Rope(torch.from_numpy(freqs).cuda(), amplitude=1.5, interleaved=il)
        yb = torch.from_numpy(y).to(torch.bfloat16).cuda()
        g = f64(nv.rope(yb, i32(pos), r, inverse=True))
        step = 1e-4
        for i in [(0, 0, 0), (1, 1, 5), (1, 0, 31), (0, 1, 40)]:
            moved = x.copy()
            moved[i] += step
            diff = ((K.rotate(moved, pos, freqs, 1.5, il) - turn) * f64(yb)).sum() / step
            # The loss is linear: the difference is exact to 1e-9; the gradient has half a BF16 step.
            assert abs(g[i] - diff) <= 2.0 ** -8 * abs(diff) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", [None, "linear", "base", "ramp", "wavelength"])
def test_rope_frequencies(nv, scaling):
    for rot, base in ((16, 1e4), (128, 5e5), (2048, 10.0)):
        got = f64(nv.rope_frequencies(rot, base, scaling, 8.0, 4096, 1.0, 4.0 if scaling == "wavelength" else 32.0))
        want = K.frequencies(scaling, rot, base, 8.0, 4096, 1.0, 4.0 if scaling == "wavelength" else 32.0)
        # pow and log in FP64 on both sides: a few steps of 2^-53, times the exponent's size (at most 16).
        assert (np.abs(got - want) <= 2.0 ** -46 * want).all()


APPEND_CASES = [
    # lens, rows, block size, heads, head_dim, rot, interleaved
    ([1], [1], 16, 1, 32, 0, False),
    ([5, 64, 33], [1, 1, 1], 16, 8, 128, 128, False),
    ([100, 7, 40], [64, 7, 1], 24, 2, 64, 32, True),
    ([0, 9, 0, 300, 3], [0, 9, 0, 257, 3], 7, 3, 96, 96, False),
    ([130], [130], 64, 10, 256, 256, True),
    ([17, 18], [17, 2], 1, 1, 160, 16, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", range(len(APPEND_CASES)))
def test_kv_append(nv, case, dt, fmt):
    """Bit for bit (R26, R27): the whole cache, also where nothing was written."""
    lens, n, bs, heads, d, rot, il = APPEND_CASES[case]
    dt, rng = TYPES[dt], np.random.default_rng(100 + case)
    nb, table, lens, start = make_batch(rng, lens, n, bs)
    rows = int(start[-1])
    c = make_cache(rng, fmt, nb, bs, heads, d)
    cache = device_cache(nv, fmt, c)
    merged = rand(rng, (rows, 2 * heads + 1, d), dt, 2.0)
    merged[rng.random(merged.shape) < 0.1] = 0.0
    k, v = merged[:, :heads], merged[:, heads + 1:]
    freqs = K.frequencies("ramp", rot, 1e6, 4.0, 2048) if rot else None
    r = nv.Rope(torch.from_numpy(freqs).cuda(), 1.0625, il) if rot else None
    with_start = (n != [1] * len(n),) if n == [1] * len(n) else (True,)
    for given in (None, rng.integers(0, 2 ** 21, size=rows) if rot else None):
        for ws in with_start + (True,):
            nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start) if ws else None, r,
                         None if given is None else i32(given))
            c = K.append(fmt, c, f64(k), f64(v), table, lens, start, freqs, 1.0625, il, given)
            same_cache(host_cache(cache, c), c)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_kv_append_borders_and_nonfinite(nv, fmt):
    """Values on and next to the borders between codes and between scales, the smallest and largest, infinities, NaN."""
    rng = np.random.default_rng(7)
    d, rows = 64, 96
    # Halves of tscale multiples hit E2M1's and E4M3's borders exactly.
    for ts in (2.0 ** -6, 0.3, 2.0 ** -120):
        x = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 5.5, 0.0, -0.0], size=(rows, 1, d)) \
            * rng.choice([1, -1], size=(rows, 1, d)) * 2.0 ** rng.integers(-12, 5, size=(rows, 1, 1))
        x[:, :, ::16] = 6.0 * rng.choice([1.0, 1.0625, 1.125, 1.1875, 70.0, 0.001], size=(rows, 1, d // 16))
        x = x.astype(np.float32)
        x[3, 0, 5], x[4, 0, 40], x[5, 0, 63], x[6] = np.inf, np.nan, -np.inf, 0.0
        x[7], x[8] = 2.0 ** -130, 3e38
        t = torch.from_numpy(x).to(torch.bfloat16).cuda()
        nb, table, lens, start = make_batch(rng, [rows], [rows], 16)
        c = make_cache(rng, fmt, nb, 16, 1, d)
        c["k_tscale"] = c["v_tscale"] = np.float32(ts) if fmt == "nvfp4" else None
        cache = device_cache(nv, fmt, c)
        freqs = K.frequencies(None, 32, 1e4)
        r = nv.Rope(torch.from_numpy(freqs).cuda())
        for rope in (None, r):
            nv.kv_append(t, t, cache, i32(table), i32(lens), i32(start), rope)
            c = K.append(fmt, c, f64(t), f64(t), table, lens, start, None if rope is None else freqs)
            same_cache(host_cache(cache, c), c)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("ts", [2.0 ** -7, 255 * 2.0 ** -14, 257 * 2.0 ** -15, 0.0078])
def test_kv_append_every_value(nv, ts, dt):
    """Every 16-bit value over seven powers of two, beside tops that choose the block's scale: each tie and its nearest
    neighbours, for tensor scales of 1, 8, 9 and 24 significant bits."""
    dt, rng = TYPES[dt], np.random.default_rng(12)
    bits = torch.arange(*(int(torch.tensor(x, dtype=dt).view(torch.int16)) for x in (2.0 ** -4, 2.0 ** 3)), dtype=torch.int16)
    x = bits.view(dt)
    tops = torch.tensor([6.0, 7.0, 8.5, 9.0, 10.5, 11.0], dtype=dt)
    n = -(-x.numel() // 15) * 15
    x = torch.cat([x, x[:n - x.numel()]]).reshape(1, -1, 15).expand(len(tops), -1, 15)
    x = torch.cat([tops[:, None, None].expand(-1, x.shape[1], 1), x], -1).reshape(-1, 16)
    x = torch.cat([x, x[:-len(x) % 8]])
    x = x.reshape(-1, 2, 64).clone().cuda()
    rows = len(x)
    nb, table, lens, start = make_batch(rng, [rows], [rows], 16)
    c = make_cache(rng, "nvfp4", nb, 16, 2, 64)
    c["k_tscale"] = c["v_tscale"] = np.float32(ts)
    cache = device_cache(nv, "nvfp4", c)
    nv.kv_append(x, -x, cache, i32(table), i32(lens), i32(start))
    c = K.append("nvfp4", c, f64(x), f64(-x), table, lens, start)
    same_cache(host_cache(cache, c), c)


@pytest.mark.gpu
@pytest.mark.parametrize("heads, d", [(1, 32), (2, 64), (8, 128), (40, 128)])
def test_kv_append_short_sequences(nv, heads, d):
    """Sequences of no, one and a few rows, many of them within a workgroup's."""
    rng = np.random.default_rng(13)
    n = rng.choice([0, 0, 0, 1, 2, 5, 40], size=200)
    lens = n + rng.integers(0, 30, size=200)
    nb, table, lens, start = make_batch(rng, list(lens), list(n), 16)
    rows = int(start[-1])
    c = make_cache(rng, "mxfp4", nb, 16, heads, d)
    cache = device_cache(nv, "mxfp4", c)
    k, v = rand(rng, (rows + 3, heads, d), torch.bfloat16), rand(rng, (rows + 3, heads, d), torch.bfloat16)
    freqs = K.frequencies(None, 32, 1e4)
    nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start), nv.Rope(torch.from_numpy(freqs).cuda()))
    c = K.append("mxfp4", c, f64(k), f64(v), table, lens, start, freqs)
    same_cache(host_cache(cache, c), c)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_kv_append_skips(nv, fmt):
    """Pages outside the cache, tokens below 0 and past the table, rows of no sequence, negative lengths."""
    rng = np.random.default_rng(8)
    nb, bs, heads, d = 5, 4, 2, 64
    table = np.array([[0, 99, 1], [-1, 2, 3], [4, 4, 4]], np.int32)
    lens, start = np.array([12, 40, 2], np.int32), np.array([2, 12, 20, 26], np.int32)  # row 2 on; 26 rows of 30
    c = make_cache(rng, fmt, nb, bs, heads, d)
    cache = device_cache(nv, fmt, c)
    k, v = rand(rng, (30, heads, d), torch.float16), rand(rng, (30, heads, d), torch.float16)
    nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
    c = K.append(fmt, c, f64(k), f64(v), table, lens, start)
    same_cache(host_cache(cache, c), c)
    for lens in ([-5, 0, -2 ** 31], [2 ** 31 - 1] * 3):
        nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
        c = K.append(fmt, c, f64(k), f64(v), table, np.array(lens, np.int64), start)
        same_cache(host_cache(cache, c), c)
    # Starts outside the rows: nothing outside the buffers is touched.
    start = np.array([-7, 5, 29, 4000], np.int32)
    lens = np.array([12, 12, 12], np.int32)
    nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
    c = K.append(fmt, c, f64(k), f64(v), table, lens, start)
    same_cache(host_cache(cache, c), c)


# lens, rows, block size, heads, group, head_dim, window
ATTEND_CASES = [
    ([1], [1], 16, 1, 1, 64, 0),
    ([1000], [1], 16, 8, 5, 128, 0),
    ([31, 32, 33, 1, 700], [1] * 5, 16, 2, 4, 128, 0),
    ([333], [1], 1, 3, 2, 96, 0),
    ([90, 4000, 257], [1, 1, 1], 24, 10, 1, 64, 0),
    ([129, 65], [1, 1], 128, 1, 16, 256, 0),
    ([200, 77], [1, 1], 16, 4, 17, 192, 0),
    ([900, 40, 2000], [1, 1, 1], 16, 4, 8, 128, 100),
    ([64, 333, 5], [5, 4, 5], 16, 2, 8, 128, 0),
    ([300, 12], [9, 12], 7, 2, 3, 96, 33),
    ([257, 100, 1], [257, 64, 1], 16, 2, 5, 128, 0),
    ([500, 0, 30], [70, 0, 30], 24, 1, 4, 64, 64),
    ([150], [150], 32, 1, 8, 256, 0),
    ([90], [80], 16, 2, 2, 192, 0),
]


def check_attention(got, q, c, fmt, table, lens, start, scale, window, left=None):
    weight = {("nvfp4", torch.bfloat16): 2.0 ** -11, ("nvfp4", torch.float16): 2.0 ** -11,
              ("mxfp4", torch.bfloat16): 2.0 ** -8, ("mxfp4", torch.float16): 2.0 ** -15}[fmt, q.dtype]
    y, bound, mine = K.attention(fmt, c, f64(q), table, lens, start, scale, window, weight)
    g = f64(got)
    h = HALF_STEP[q.dtype]
    nan = np.isnan(y) | np.isnan(bound)
    if q.dtype == torch.float16:
        # Half a step above FP16's largest number, 65504 + 16, rounding gives infinity: that is the result there.
        over = ~nan & (np.abs(y) + np.abs(bound) >= 65520)
        assert (np.isinf(g) | ~over)[mine].all() and (np.sign(g) == np.sign(y))[over & mine[:, None, None]].all()
        y, g = np.where(over, 0.0, y), np.where(over, 0.0, g)
    off = np.abs(g - y) - (bound + h * (np.abs(y) + bound) + TINY[q.dtype])
    assert np.array_equal(np.isnan(g[mine]), nan[mine])
    assert not (off[mine] > 0)[~nan[mine]].any(), f"{np.nanmax(off[mine])} over, worst at {np.unravel_index(np.nanargmax(off), off.shape)}"
    if left is not None:
        assert (g[~mine] == left).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", range(len(ATTEND_CASES)))
def test_kv_attention(nv, case, dt, fmt):
    lens, n, bs, heads, g, d, window = ATTEND_CASES[case]
    dt, rng = TYPES[dt], np.random.default_rng(200 + case)
    nb, table, lens, start = make_batch(rng, lens, n, bs)
    rows = int(start[-1])
    c = make_cache(rng, fmt, nb, bs, heads, d)
    cache = device_cache(nv, fmt, c)
    q = rand(rng, (rows + 2, heads * g + 1, d), dt)[:, 1:]
    out = torch.full((rows + 2, heads * g, d), 3.0, dtype=dt, device="cuda")
    args = (cache, i32(table), i32(lens))
    got = nv.kv_attention(q, *args, i32(start), window=window or None, out=out)
    assert got is out
    check_attention(got, q, c, fmt, table, lens, start, d ** -0.5, window, left=3.0)
    again = nv.kv_attention(q[:rows], *args, i32(start), window=window or None)
    assert torch.equal(again, nv.kv_attention(q[:rows], *args, i32(start), window=window or None))
    check_attention(again, q[:rows], c, fmt, table, lens, start, d ** -0.5, window)
    if n == [1] * len(n):
        assert torch.equal(again, nv.kv_attention(q[:rows], *args, window=window or None))
    sharp = nv.kv_attention(q[:rows], *args, i32(start), scale=-1.75, window=window or None)
    check_attention(sharp, q[:rows], c, fmt, table, lens, start, -1.75, window)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("per", [1, 3, 40])
def test_kv_attention_hidden_values(nv, fmt, per):
    """NaN blocks, and infinities in the query, reach the rows that see them and no other: tokens above a row, below its
    window, behind the length, in pages outside the cache."""
    rng = np.random.default_rng(300 + per)
    heads, g, d, bs, window = 2, 4, 64, 16, 50
    lens, n = [130, 200, 61], [per, per, per]
    nb, table, lens, start = make_batch(rng, lens, n, bs)
    c = make_cache(rng, fmt, nb, bs, heads, d)
    q = rand(rng, (3 * per, heads * g, d), torch.float16)
    nan = 0x7F if fmt == "nvfp4" else 255

    def poison(name, s, t, h, block):
        c[name][table[s, t // bs], t % bs, h, block] = nan
    # Behind every length and in every spare slot.
    for s in range(3):
        for t in range(int(lens[s]), -(-int(lens[s]) // bs) * bs):
            c["v_scales"][table[s, t // bs], t % bs] = nan
            c["k_scales"][table[s, t // bs], t % bs] = nan
    poison("v_scales", 0, 129, 0, 1)                       # the last token: only its own row sees it
    poison("v_scales", 0, 130 - per, 1, 0)                 # the first of the call's tokens
    poison("v_scales", 1, 200 - per - window + 1, 0, 1)    # the first row's window's first token
    poison("v_scales", 1, 3, 1, 0)                         # below every window
    poison("k_scales", 2, 60, 1, 0)
    if fmt == "mxfp4":
        c["v_scales"][table[2, 2], 5, 0, 0] = 254          # beyond FP32's range: counts as NaN
        c["v_scales"][table[2, 2], 6, 1, 1] = 252          # still a number
        c["v_codes"][table[2, 2], 6, 1] = 0x11
    table[2, 0] = nb + 5                                   # a page outside the cache
    cache = device_cache(nv, fmt, c)
    for w in (window, 0):
        got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=w or None)
        check_attention(got, q, c, fmt, table, lens, start, d ** -0.5, w)
        assert np.isnan(f64(got)).any() and np.isfinite(f64(got)).any()
    q[0, 0, 5], q[1 % (3 * per), 3, 7] = float("inf"), float("nan")
    got = f64(nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=window))
    q[0, 0, 5] = q[1 % (3 * per), 3, 7] = 0.0
    clean = f64(nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=window))
    same = np.ones(got.shape[:2], bool)
    same[0, 0] = same[1 % (3 * per), 3] = False
    assert np.array_equal(got[same], clean[same], equal_nan=True)
    assert np.isnan(got[1 % (3 * per), 3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_kv_attention_values_and_scales_far_apart(nv, fmt):
    """Queries near the type's largest and smallest numbers, block scales at both ends of their range, tensor scales of
    0, tiny and negative: the same formula."""
    rng = np.random.default_rng(9)
    heads, g, d, bs = 1, 4, 64, 16
    nb, table, lens, start = make_batch(rng, [100, 33], [2, 1], bs)
    for dt in (torch.bfloat16, torch.float16):
        for size, kt in ((1e4, 2.0 ** -14), (1e-4, 4.0), (2.0 ** -12, 0.0), (1.0, -0.25)):
            c = make_cache(rng, fmt, nb, bs, heads, d)
            if fmt == "nvfp4":
                c["k_scales"] = rng.choice([0x00, 0x01, 0x08, 0x30, 0x50, 0x7E], size=c["k_scales"].shape).astype(np.uint8)
                c["v_scales"] = rng.choice([0x00, 0x01, 0x30, 0x7E], size=c["v_scales"].shape).astype(np.uint8)
                c["k_tscale"] = np.float32(kt * 2.0 ** -7)
            else:
                c["k_scales"] = rng.choice([90, 110, 126, 127], size=c["k_scales"].shape).astype(np.uint8)
                c["v_scales"] = rng.choice([0, 60, 127, 200], size=c["v_scales"].shape).astype(np.uint8)
            cache = device_cache(nv, fmt, c)
            q = rand(rng, (3, heads * g, d), dt, size)
            scale = 0.125 / size if fmt == "mxfp4" else 0.125
            got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale)
            y = f64(got)
            if dt == torch.float16 and fmt == "mxfp4":
                continue                                    # 2^73 is no FP16 number
            check_attention(got, q, c, fmt, table, lens, start, scale, 0)
            assert np.isfinite(y).all()


@pytest.mark.gpu
def test_kv_attention_many_sequences(nv):
    """More sequences than a wavefront and a workgroup have lanes, empty ones and empty lengths among them; rows before
    the first and behind the last are left."""
    rng = np.random.default_rng(10)
    for seqs, most in ((65, 40), (900, 9), (1100, 3)):
        n = rng.integers(0, 2, size=seqs) * rng.integers(1, 3, size=seqs)
        lens = np.where(rng.random(seqs) < 0.1, 0, n + rng.integers(0, most, size=seqs))
        nb, table, lens, start = make_batch(rng, lens.tolist(), n.tolist(), 4)
        start = (start + 3).astype(np.int32)
        rows = int(start[-1]) + 2
        c = make_cache(rng, "nvfp4", nb, 4, 2, 64)
        cache = device_cache(nv, "nvfp4", c)
        q = rand(rng, (rows, 4, 64), torch.float16)
        out = torch.full_like(q, 9.0)
        nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), out=out)
        check_attention(out, q, c, "nvfp4", table, lens, start, 0.125, 0, left=9.0)
        k, v = rand(rng, (rows, 2, 64), torch.float16), rand(rng, (rows, 2, 64), torch.float16)
        nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
        same_cache(host_cache(cache, c), K.append("nvfp4", c, f64(k), f64(v), table, lens, start))
    # The same through the kernel for many rows.
    seqs = 1100
    n = np.where(rng.random(seqs) < 0.97, 0, rng.integers(1, 700, size=seqs))
    n[5], n[6] = 3000, 0
    lens = n + rng.integers(0, 3, size=seqs)
    nb, table, lens, start = make_batch(rng, lens.tolist(), n.tolist(), 32)
    c = make_cache(rng, "mxfp4", nb, 32, 1, 64)
    q = rand(rng, (int(start[-1]), 8, 64), torch.bfloat16)
    cache = device_cache(nv, "mxfp4", c)
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=20)
    check_attention(got, q, c, "mxfp4", table, lens, start, 0.125, 20)


@pytest.mark.gpu
def test_kv_ops_bad_device_data(nv):
    """Lengths, starts and pages that make no sense: nothing faults, rows that belong to no sequence stay, and sound
    sequences beside them are right."""
    rng = np.random.default_rng(11)
    nb, bs, heads, d = 40, 16, 2, 64
    c = make_cache(rng, "nvfp4", nb, bs, heads, d)
    cache = device_cache(nv, "nvfp4", c)
    table = rng.integers(-50, 100, size=(6, 8)).astype(np.int32)
    for rows, g in ((12, 2), (64, 8)):
        q = rand(rng, (rows, heads * g, d), torch.bfloat16)
        k = rand(rng, (rows, heads, d), torch.bfloat16)
        for lens in ([-1, 0, 2 ** 31 - 1, -2 ** 31, 50, 129], [5, 128, 3000, 1, 0, 7]):
            lens = np.array(lens, np.int64)
            start = np.sort(rng.integers(-3, rows + 4, size=7)).astype(np.int32)
            out = torch.full_like(q, 2.0)
            nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), out=out)
            check_attention(out, q, c, "nvfp4", table, lens, start, d ** -0.5, 0, left=2.0)
            for start in ([9, 3, 9, 0, 2 ** 31 - 1, -7, 5], [rows] * 7, [0, rows, 0, rows, 0, rows, 0]):
                nv.kv_attention(q, cache, i32(table), i32(lens), i32(start))
                nv.kv_append(k, k, cache, i32(np.full_like(table, -1)), i32(lens), i32(start))
    same_cache(host_cache(cache, c), c)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_kv_ops_beyond_32_bits(nv, fmt):
    """Pages whose codes lie more than 2^32 bytes from the start, and the cache's last page."""
    rng = np.random.default_rng(12)
    bs, heads, d = 64, 8, 128
    nb = 2 ** 32 // (bs * heads * d // 2) + 40
    shape = (nb, bs, heads)
    sc = d // K.GROUP[fmt]
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    t = [torch.empty((*shape, w), dtype=torch.uint8, device="cuda") for w in (d // 2, sc, d // 2, sc)]
    ts = torch.full((1,), 0.02, device="cuda") if fmt == "nvfp4" else None
    cache = nv.KVCache(*t, ts, ts, fmt)
    pages = np.array([nb - 1, 3, nb - 20, nb - 39, 7, nb - 2], np.int32)
    for n, per in (([6 * 64 - 5], 6 * 64 - 5), ([300], 300)):
        table = pages[None]
        rows = n[0]
        k, v = rand(rng, (rows, heads, d), torch.bfloat16), rand(rng, (rows, heads, d), torch.bfloat16)
        lens, start = np.array(n, np.int32), np.array([0, rows], np.int32)
        nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
        small = {"k_codes": t[0], "k_scales": t[1], "v_codes": t[2], "v_scales": t[3]}
        small = {name: x[torch.from_numpy(pages).long().cuda()].cpu().numpy() for name, x in small.items()}
        small.update(k_tscale=np.float32(0.02) if ts is not None else None, v_tscale=np.float32(0.02) if ts is not None else None)
        near = np.arange(6, dtype=np.int32)[None]
        want = K.append(fmt, small, f64(k), f64(v), near, lens, start)
        same_cache(small, want)
        for qrows in (1, 40):
            q = rand(rng, (qrows, heads * 2, d), torch.bfloat16)
            st = np.array([0, qrows], np.int32)
            got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(st))
            check_attention(got, q, small, fmt, near, lens, st, d ** -0.5, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_kv_ops_in_a_row(nv, fmt):
    """A prompt in two chunks and then single tokens, as a layer runs them: queries turned, keys and values appended,
    attention.  Every step against the oracle's cache and formula; the gather sees the same cache."""
    rng = np.random.default_rng(13)
    heads, g, d, bs, seqs = 2, 3, 64, 16, 3
    freqs = K.frequencies("ramp", 32, 1e4, 4.0, 64)
    rope = nv.Rope(nv.rope_frequencies(32, 1e4, "ramp", 4.0, 64), amplitude=1.125)
    ts = torch.full((1,), 0.01, device="cuda") if fmt == "nvfp4" else None
    cache = nv.KVCache.zeros(40, bs, heads, d, fmt, ts, ts)
    c = {n: getattr(cache, n).cpu().numpy() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    c.update(k_tscale=None if ts is None else np.float32(0.01), v_tscale=None if ts is None else np.float32(0.01))
    table = rng.permutation(40)[:seqs * 8].reshape(seqs, 8).astype(np.int32)
    lens = np.zeros(seqs, np.int32)
    for n in ([60, 7, 33], [20, 30, 1], [1, 1, 1], [1, 1, 1], [2, 0, 3]):
        lens = lens + np.array(n, np.int32)
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        qkv = rand(rng, (int(start[-1]), heads * (g + 2), d), torch.bfloat16)
        q, k, v = qkv.split([heads * g, heads, heads], 1)
        pos = np.concatenate([np.arange(m - j, m) for m, j in zip(lens, n)])
        turned = nv.rope(q, i32(pos), rope)
        nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start), rope)
        got = nv.kv_attention(turned, cache, i32(table), i32(lens), i32(start))
        c = K.append(fmt, c, f64(k), f64(v), table, lens, start, freqs, 1.125)
        # nv.rope_frequencies' powers differ from the oracle's in their last bits: a key's FP32 rounding may too.
        mine = host_cache(cache, c)
        assert all((mine[x] != c[x]).mean() < 1e-3 for x in ("k_codes", "k_scales"))
        assert np.array_equal(mine["v_codes"], c["v_codes"]) and np.array_equal(mine["v_scales"], c["v_scales"])
        check_attention(got, turned, mine, fmt, table, lens, start, d ** -0.5, 0)
    out = torch.zeros((int(lens.sum()), heads, d), dtype=torch.float16, device="cuda")
    dst = np.concatenate([[0], np.cumsum(lens)[:-1]])
    nv.kv_gather(cache.k_codes, cache.k_scales, cache.k_tscale, i32(table), i32(lens), i32(dst), out, fmt=fmt)
    vals = K.values(fmt, mine["k_codes"], mine["k_scales"], mine["k_tscale"])
    for s in range(seqs):
        t = np.arange(lens[s])
        want = vals[table[s, t // bs], t % bs]
        assert np.abs(f64(out)[dst[s]:dst[s] + lens[s]] - want).max() <= 2.0 ** -11 * np.abs(want).max()


@pytest.mark.gpu
def test_kv_ops_graph_and_streams(nv):
    """Captured once and replayed with other lengths and inputs, between eager calls; on another stream than the current
    one at creation; two calls at once on two streams with their own workspaces."""
    rng = np.random.default_rng(14)
    heads, g, d, bs, seqs, rows = 2, 4, 128, 16, 4, 8
    table = rng.permutation(64)[:seqs * 16].reshape(seqs, 16).astype(np.int32)
    c = make_cache(rng, "nvfp4", 64, bs, heads, d)
    freqs = torch.from_numpy(K.frequencies(None, d, 1e4)).cuda()
    rope = nv.Rope(freqs)
    q, k, v = (rand(rng, (rows, h, d), torch.bfloat16) for h in (heads * g, heads, heads))
    lens, start, pos = i32([100, 7, 200, 50]), i32([0, 3, 4, 7, 8]), i32(np.arange(rows))
    tab = i32(table)

    def step(cache):
        turned = nv.rope(q, pos, rope)
        nv.kv_append(k, v, cache, tab, lens, start, rope)
        return nv.kv_attention(turned, cache, tab, lens, start)
    eager, captured = device_cache(nv, "nvfp4", c), device_cache(nv, "nvfp4", c)
    step(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(captured)
    for i in range(4):
        lens.copy_(i32([100 + i, 7 + 3 * i, 200 - i, 50 + 11 * i]))
        q.copy_(rand(rng, q.shape, q.dtype))
        k.copy_(rand(rng, k.shape, k.dtype))
        want = step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        same_cache(host_cache(captured, c), host_cache(eager, c))
    side = [torch.cuda.Stream() for _ in range(2)]
    want = step(eager)
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in side:
            with torch.cuda.stream(s):
                got.append(nv.kv_attention(nv.rope(q, pos, rope), eager, tab, lens, start))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)


@pytest.mark.gpu
def test_kv_ops_binding_refusals(nv):
    z = torch.zeros
    cache = nv.KVCache.zeros(4, 16, 2, 64, "mxfp4")
    q, kv = z((3, 4, 64), dtype=torch.float16, device="cuda"), z((3, 2, 64), dtype=torch.float16, device="cuda")
    tab, lens = z((3, 2), dtype=torch.int32, device="cuda"), z(3, dtype=torch.int32, device="cuda")
    rope = nv.Rope(z(16, dtype=torch.float64, device="cuda"))
    wide = nv.Rope(z(40, dtype=torch.float64, device="cuda"))
    bad = [
        lambda: nv.KVCache.zeros(4, 16, 2, 48, "mxfp4"), lambda: nv.KVCache.zeros(4, 16, 2, 64, "nvfp4"),
        lambda: nv.KVCache.zeros(4, 16, 2, 64, "int4"),
        lambda: nv.KVCache(cache.k_codes, cache.k_scales, cache.v_codes[:2], cache.v_scales, fmt="mxfp4"),
        lambda: nv.KVCache(cache.k_codes, cache.k_codes, cache.v_codes, cache.v_scales, fmt="mxfp4"),
        lambda: nv.KVCache(cache.k_codes.cpu(), cache.k_scales, cache.v_codes, cache.v_scales, fmt="mxfp4"),
        lambda: nv.Rope(z(12, dtype=torch.float64, device="cuda")), lambda: nv.Rope(z(16, device="cuda")),
        lambda: nv.rope_frequencies(20), lambda: nv.rope_frequencies(32, scaling="other"),
        lambda: nv.rope(q.float(), lens, rope), lambda: nv.rope(q.cpu(), lens, rope), lambda: nv.rope(q[0], lens, rope),
        lambda: nv.rope(q, lens[:2], rope), lambda: nv.rope(q, lens, wide), lambda: nv.rope(q, lens, rope, out=q.bfloat16()),
        lambda: nv.rope(q.transpose(1, 2), lens, rope), lambda: nv.rope(q, lens, rope, out=q[:2]),
        lambda: nv.kv_append(kv, kv.bfloat16(), cache, tab, lens), lambda: nv.kv_append(q, q, cache, tab, lens),
        lambda: nv.kv_append(kv, kv, cache, tab[:2], lens[:2]), lambda: nv.kv_append(kv, kv, cache, tab, lens[:2]),
        lambda: nv.kv_append(kv, kv, cache, tab, lens, row_start=lens), lambda: nv.kv_append(kv, kv, cache, tab.long(), lens),
        lambda: nv.kv_append(kv, kv, cache, tab, lens, positions=lens), lambda: nv.kv_append(kv, kv, cache, tab, lens, rope=wide),
        lambda: nv.kv_attention(q[:, :3], cache, tab, lens), lambda: nv.kv_attention(q, cache, tab, lens, window=0),
        lambda: nv.kv_attention(q, cache, tab, lens, out=q[:2]), lambda: nv.kv_attention(q, cache, tab, lens.long()),
        lambda: nv.kv_attention(q, cache, tab, lens, row_start=lens),
        lambda: nv.kv_attention(q.transpose(0, 1).contiguous().transpose(0, 1)[..., :32], cache, tab, lens),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was not refused")
    small = nv.KVCache.zeros(4, 16, 2, 32, "mxfp4")
    with pytest.raises(ValueError):
        nv.kv_attention(q[..., :32].contiguous(), small, tab, lens)
    with pytest.raises(nv.NVFP4Error):
        nv.kv_attention(q, cache, tab, lens, workspace=z(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        nv.rope(z((3, 4, 68), dtype=torch.float16, device="cuda")[..., :64], lens, rope)      # strides not multiples of 8
    # Nothing to do.
    assert nv.kv_attention(q[:0], cache, tab[:0], lens[:0]).shape == (0, 4, 64)
    nv.kv_append(kv[:0], kv[:0], cache, tab, lens, row_start=z(4, dtype=torch.int32, device="cuda"))
    assert nv.rope(q[:0], lens[:0], rope).shape == (0, 4, 64)
