"""The E4M3 operators with block scales: refusals of the C entry points and the binding (CPU), and the HIP kernels
against the float64 oracle (GPU)."""
import math
import os

import numpy as np
import pytest
import torch

from nvfp4_weight_only_amd import binding as B
from nvfp4_weight_only_amd import build as BUILD
from nvfp4_weight_only_amd import workloads as WL
from oracle import fp8_oracle as F

U = 2.0 ** -24      # half a step of FP32, relative
EPS = 1e-6


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
# CPU: the oracle's encoder, and what the entry points refuse.
# ---------------------------------------------------------------------------
def test_fp8_oracle_encoder_matches_torch():
    grid = F._GRID
    q = np.concatenate([grid, F._MID, F._MID * (1 + 2.0 ** -20), F._MID * (1 - 2.0 ** -20),
                        np.random.default_rng(0).uniform(-448, 448, 4096)])
    q = np.concatenate([q, -q])
    want = torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.encode(q.astype(np.float32).astype(np.float64)), want)


# Fake, never-dereferenced device addresses: validation fails before any HIP call.
A, C, D, E, G, H, W = (i * 0x10000000 for i in range(1, 8))
BIG = 2 ** 62


def test_fp8_quantize_validation(L):
    q = L.nvfp4_fp8_quantize
    assert q(A, 1, 4, 128, 2, C, D, None) == B.ERR_UNSUPPORTED          # neither 1 nor 128 rows
    assert q(A, 1, 4, 120, 1, C, D, None) == B.ERR_SHAPE                # k % 16 != 0
    assert q(A, 1, 4, 0, 1, C, D, None) == B.ERR_SHAPE
    assert q(A, -1, 4, 128, 1, C, D, None) == B.ERR_SHAPE and q(A, 1, -1, 128, 1, C, D, None) == B.ERR_SHAPE
    assert q(A, 1, BIG, 128, 1, C, D, None) == B.ERR_SHAPE
    assert q(A, 2 ** 20, 2 ** 20, 16, 1, C, D, None) == B.ERR_UNSUPPORTED
    assert q(None, 0, 4, 128, 1, None, None, None) == B.OK and q(None, 1, 0, 128, 128, None, None, None) == B.OK
    assert q(None, 1, 4, 128, 1, C, D, None) == B.ERR_NULL and q(A, 1, 4, 128, 1, C, None, None) == B.ERR_NULL
    assert q(A + 8, 1, 4, 128, 1, C, D, None) == B.ERR_ALIGN and q(A, 1, 4, 128, 1, C, D + 4, None) == B.ERR_ALIGN
    assert q(A, 1, 4, 128, 1, A + 512, D, None) == B.ERR_ALIAS          # codes overlap w
    assert q(A, 1, 4, 128, 1, C, C + 256, None) == B.ERR_ALIAS          # scales overlap codes


def test_rmsnorm_fp8_validation(L):
    f = L.nvfp4_rmsnorm_fp8
    assert f(A, None, C, EPS, 4, 100, None, D, E, None) == B.ERR_SHAPE
    assert f(A, None, C, EPS, -1, 128, None, D, E, None) == B.ERR_SHAPE
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert f(A, None, C, eps, 4, 128, None, D, E, None) == B.ERR_UNSUPPORTED
    assert f(None, None, None, EPS, 0, 128, None, None, None, None) == B.OK
    assert f(A, None, None, EPS, 4, 128, None, D, E, None) == B.ERR_NULL
    assert f(A, G, C, EPS, 4, 128, None, D, E, None) == B.ERR_NULL       # residual without its output
    assert f(A, None, C, EPS, 4, 128, G, D, E, None) == B.ERR_NULL       # and the reverse
    assert f(A, G, C + 2, EPS, 4, 128, H, D, E, None) == B.ERR_ALIGN
    assert f(A, G, C, EPS, 4, 128, G + 16, D, E, None) == B.ERR_ALIAS    # the residual's buffer, but shifted
    assert f(A, G, C, EPS, 4, 128, A, D, E, None) == B.ERR_ALIAS         # over x
    assert f(A, G, C, EPS, 4, 128, H, H, E, None) == B.ERR_ALIAS         # two outputs
    assert f(A, G, C, EPS, 4, 128, G, G, E, None) == B.ERR_ALIAS         # in place, codes over the residual


def test_silu_mul_fp8_validation(L):
    f = L.nvfp4_silu_mul_fp8
    assert f(A, 4, 24, C, D, None) == B.ERR_SHAPE and f(A, 4, 0, C, D, None) == B.ERR_SHAPE
    assert f(None, 0, 128, None, None, None) == B.OK
    assert f(None, 4, 128, C, D, None) == B.ERR_NULL
    assert f(A, 4, 128, C + 8, D, None) == B.ERR_ALIGN
    assert f(A, 4, 128, A + 4 * 512 - 16, D, None) == B.ERR_ALIAS        # codes over the last up columns


def test_fp8_linear_validation(L):
    f, wb = L.nvfp4_fp8_linear, L.nvfp4_fp8_linear_workspace_bytes
    assert f(A, C, 4, 64, 24, D, E, G, None, 0, None) == B.ERR_SHAPE     # k % 16 != 0
    assert f(A, C, 4, 0, 128, D, E, G, None, 0, None) == B.ERR_SHAPE
    assert f(A, C, -1, 64, 128, D, E, G, None, 0, None) == B.ERR_SHAPE
    assert f(A, C, 4, BIG, 128, D, E, G, None, 0, None) == B.ERR_SHAPE
    assert f(A, C, 4, 64, 128, D, E, G, None, -1, None) == B.ERR_SHAPE
    assert f(None, None, 0, 64, 128, D, E, None, None, 0, None) == B.OK  # m = 0
    assert f(None, None, 0, 64, 128, None, E, None, None, 0, None) == B.ERR_NULL
    assert f(A, None, 4, 64, 128, D, E, G, None, 0, None) == B.ERR_NULL
    assert f(A, C + 4, 4, 64, 128, D, E, G, None, 0, None) == B.ERR_ALIGN
    assert f(A, C, 4, 64, 128, D, E, G, W + 8, 1 << 20, None) == B.ERR_ALIGN
    assert f(A, C, 4, 64, 128, D, E, A + 496, None, 0, None) == B.ERR_ALIAS
    assert f(A, C, 4, 64, 128, D, E, D, None, 0, None) == B.ERR_ALIAS
    assert wb(4, 64, 24) == -1 and wb(-1, 64, 128) == -1 and wb(4, 0, 128) == -1 and wb(0, 64, 128) == 0


def test_fp8_linear_grouped_validation(L):
    f, wb = L.nvfp4_fp8_linear_grouped, L.nvfp4_fp8_linear_grouped_workspace_bytes
    need = wb(2, 2, 2)

    def args(xq=A, t=2, topk=2, route=H, e=2, n=64, k=128, wq=D, y=G, ws=W, wsb=need):
        return (xq, C, t, topk, route, e, n, k, wq, E, y, ws, wsb, None)
    assert wb(-1, 1, 1) == -1 and wb(1, 0, 1) == -1 and wb(1, 1, 0) == -1 and wb(BIG, 4, 1) == -1
    assert f(*args(topk=0)) == B.ERR_SHAPE and f(*args(e=0)) == B.ERR_SHAPE and f(*args(k=40)) == B.ERR_SHAPE
    assert f(*args(n=0)) == B.ERR_SHAPE and f(*args(t=-1)) == B.ERR_SHAPE and f(*args(wsb=need - 16)) == B.ERR_SHAPE
    assert f(*args(ws=None)) == B.ERR_NULL and f(*args(wq=None)) == B.ERR_NULL and f(*args(route=None)) == B.ERR_NULL
    assert f(*args(route=H + 2)) == B.ERR_ALIGN and f(*args(ws=W + 8)) == B.ERR_ALIGN
    assert f(*args(ws=H)) == B.ERR_ALIAS and f(*args(y=A)) == B.ERR_ALIAS and f(*args(ws=G)) == B.ERR_ALIAS
    assert f(*args(xq=None, t=0, y=None, ws=None, wsb=0)) == B.OK


# ---------------------------------------------------------------------------
# GPU.
# ---------------------------------------------------------------------------
def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(bits):
    return WL.f32_from_bf16_bits(bits).astype(np.float64)


def host(t):
    return t.double().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def same_scales(got, want):
    return np.array_equal(host(got).view(np.uint32), np.where(np.isnan(want), np.float32("nan"), want)
                          .astype(np.float32).view(np.uint32))


def crafted():
    """One row of 128: a tie on every E4M3 midpoint (amax 448 or a power of two times it), zeros, extremes."""
    mids = np.concatenate([F._MID, [448.0, -448.0]])
    rows = {"ties": mids, "ties, other signs": -mids, "zeros": np.zeros(16), "negative zeros": -np.zeros(16),
            "huge": [3.0e38, -1e38, 1.0, -1e-30] * 4, "subnormal": [1e-40, -2e-39, 3e-41, 0.0] * 4,
            "smallest": [9.2e-41, -9.2e-41] * 8, "infinity": [np.inf] + [1.0] * 15, "nan": [1.0] * 15 + [np.nan]}
    out = {}
    for name, v in rows.items():
        r = np.zeros(-(-len(v) // 16) * 16, dtype=np.float32)
        r[:len(v)] = v
        out[name] = WL.bf16_bits_from_f32(r[None])
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("shape,block_rows", [
    ((1, 16), 1), ((1, 16), 128), ((3, 128), 1), ((8, 5120), 1), ((130, 272), 1), ((130, 272), 128), ((257, 144), 128),
    ((1, 40000), 1), ((700, 8192), 1), ((3, 100, 208), 128), ((2, 128, 128), 128), ((3, 5, 208), 1)])
def test_fp8_quantize_bit_exact(nv, shape, block_rows):
    bits = WL.normal_bf16(shape, 0.02, 100 + shape[-1])
    codes, scales = nv.fp8_quantize(bf16(bits), block_rows)
    rc, rs = F.quantize(f64(bits), block_rows)
    assert codes.shape == rc.shape and scales.shape == rs.shape
    assert same_scales(scales, rs) and np.array_equal(host(codes), rc)


# More than 32768 blocks of 1 x 128, so several per thread: 32 .. 63 blocks a row (two, with one scalar division per
# workgroup), 64 and more and fewer than 16 (four, with and without), 16 .. 31 (one).
MANY_BLOCKS = [(2048, 5120), (1100, 4112), (900, 8208), (4200, 1040), (33000, 16), (2100, 2064)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", MANY_BLOCKS)
def test_fp8_quantize_many_blocks(nv, m, k):
    bits = WL.normal_bf16((m, k), 0.02, 110 + k)
    codes, scales = nv.fp8_quantize(bf16(bits))
    rc, rs = F.quantize(f64(bits), 1)
    assert same_scales(scales, rs) and np.array_equal(host(codes), rc)


@pytest.mark.gpu
@pytest.mark.parametrize("block_rows", [1, 128])
def test_fp8_quantize_crafted(nv, block_rows):
    for name, bits in crafted().items():
        codes, scales = nv.fp8_quantize(bf16(bits), block_rows)
        rc, rs = F.quantize(f64(bits), block_rows)
        assert same_scales(scales, rs), name
        assert np.array_equal(host(codes), rc), name


@pytest.mark.gpu
def test_fp8_quantize_random_bits(nv):
    """Every exponent: rows of random finite BF16 patterns against amax of every size."""
    rng = np.random.default_rng(7)
    bits = rng.integers(0, 1 << 16, size=(512, 256)).astype(np.uint16)
    bits[(bits & 0x7F80) == 0x7F80] &= 0xBFFF
    bits &= np.uint16(0x8000) | (np.linspace(0x100, 0x7F7F, 512).astype(np.uint16)[:, None])
    codes, scales = nv.fp8_quantize(bf16(bits), 1)
    rc, rs = F.quantize(f64(bits), 1)
    assert same_scales(scales, rs) and np.array_equal(host(codes), rc)


NORM_CASES = [(1, 16), (5, 128), (7, 400), (8, 5120), (300, 1024), (3, 8192), (3, 8208), (2, 32768), (2, 40016)]


def norm_tolerance(k):
    """Relative error of a scale: the sum of squares is a chain of at most 8 additions per piece and ceil(k / 8192)
    or 4 pieces a thread, 6 in the wavefront and 16 across them (u each, halved by the root); the division by k, the
    sum with eps, root and reciprocal and two more factors, u each."""
    chain = 8 * max(4, -(-k // 8192)) + 22
    return (chain / 2 + 6) * U * 2


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", NORM_CASES)
@pytest.mark.parametrize("mode", ["plain", "residual", "in place"])
def test_rmsnorm_fp8(nv, m, k, mode):
    xb, rb = WL.normal_bf16((m, k), 1.0, 200 + k), WL.normal_bf16((m, k), 4.0, 201 + k)
    gb = WL.normal_bf16((k,), 1.0, 202 + k)
    x, g, r = bf16(xb), bf16(gb), bf16(rb)
    h = f64(xb)
    if mode == "plain":
        codes, scales, h_out = nv.rmsnorm_fp8(x, g, EPS)
        assert h_out is None
    else:
        hb = WL.bf16_bits_from_f32(WL.f32_from_bf16_bits(xb) + WL.f32_from_bf16_bits(rb))
        h = f64(hb)
        codes, scales, h_out = nv.rmsnorm_fp8(x, g, EPS, residual=r, residual_out=r if mode == "in place" else None)
        assert np.array_equal(host(h_out), h)
        assert mode == "in place" or np.array_equal(host(r), f64(rb))
        assert (h_out.data_ptr() == r.data_ptr()) == (mode == "in place")
    rc, rs = F.norm(h, f64(gb), EPS)
    assert np.array_equal(host(codes), rc)
    assert np.all(np.abs(host(scales) - rs) <= norm_tolerance(k) * rs)


# More than 512 rows: three pieces a thread, in workgroups of one wavefront and of several.
@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(600, 16), (700, 400), (513, 5120), (515, 1552)])
@pytest.mark.parametrize("mode", ["plain", "residual", "in place"])
def test_rmsnorm_fp8_many_rows(nv, m, k, mode):
    test_rmsnorm_fp8(nv, m, k, mode)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(6, 384), (600, 384), (530, 5120), (6, 40960)])
@pytest.mark.parametrize("mode", ["plain", "residual", "in place"])
def test_rmsnorm_fp8_odd_rows_everywhere(nv, m, k, mode):
    """The odd rows below in every kernel: rows of zeros, a block of zeros, a square that overflows, infinities (one of
    them made by the residual's addition) and NaN change their own rows only."""
    xb, rb, gb = WL.normal_bf16((m, k), 1.0, 320 + k), WL.normal_bf16((m, k), 1.0, 321 + k), WL.normal_bf16((k,), 1.0, 322 + k)
    xb[0], rb[0], xb[m - 1, 128:256], rb[m - 1, 128:256] = 0, 0, 0, 0
    xb[1, k - 1] = WL.bf16_bits_from_f32(np.float32([3e38]))[0]
    xb[2, 7], xb[3, 300] = 0x7F80, 0x7FC0
    xb[4, 9], rb[4, 9] = 0x7F00, 0x7F00 if mode != "plain" else 0       # 2^127 twice: infinite when added
    x, r, g = bf16(xb), bf16(rb), bf16(gb)
    h = f64(xb)
    if mode == "plain":
        codes, scales, _ = nv.rmsnorm_fp8(x, g, EPS)
    else:
        want = (x.float() + r.float()).bfloat16()
        h = host(want)
        codes, scales, out = nv.rmsnorm_fp8(x, g, EPS, residual=r, residual_out=r if mode == "in place" else None)
        assert torch.equal(out.nan_to_num(1e30, 2e30), want.nan_to_num(1e30, 2e30))
    codes, scales = host(codes), host(scales)
    assert not codes[0].any() and not scales[0].any()
    assert not codes[m - 1, 128:256].any() and scales[m - 1, 1] == 0
    for row in (1, 2, 3, 4):
        assert np.all(codes[row] == 0x7F) and np.isnan(scales[row]).all(), row
    rc, rs = F.norm(h[5:], f64(gb), EPS)
    assert np.array_equal(codes[5:], rc)
    assert np.all(np.abs(scales[5:] - rs) <= norm_tolerance(k) * rs)


@pytest.mark.gpu
def test_rmsnorm_fp8_odd_rows(nv):
    """Zero rows and blocks, a row whose squares overflow FP32, infinities and NaN: only their own rows change."""
    k = 384
    xb = WL.normal_bf16((6, k), 1.0, 300)
    xb[0] = 0
    xb[1, 128:256] = 0
    xb[2, 5] = WL.bf16_bits_from_f32(np.float32([3e38]))[0]
    xb[3, 7] = 0x7F80
    xb[4, 300] = 0x7FC0
    g = np.ones(k, dtype=np.float32)
    codes, scales, _ = nv.rmsnorm_fp8(bf16(xb), bf16(WL.bf16_bits_from_f32(g)), EPS)
    codes, scales = host(codes), host(scales)
    rc, rs = F.norm(f64(xb), g.astype(np.float64), EPS)
    assert not codes[0].any() and not scales[0].any() and not codes[1, 128:256].any() and scales[1, 1] == 0
    for row in (1, 5):
        assert np.array_equal(codes[row], rc[row])
        assert np.all(np.abs(scales[row] - rs[row]) <= norm_tolerance(k) * rs[row])
    for row in (2, 3, 4):
        assert np.all(codes[row] == 0x7F) and np.isnan(scales[row]).all()


# Standard deviations of h and of the weight whose products overflow FP32, are subnormal, or are 0 there.
@pytest.mark.gpu
@pytest.mark.parametrize("h_exp,g_exp", [(50, 90), (-70, -70), (-100, -90), (-100, -20), (-40, -88)])
@pytest.mark.parametrize("m,k", [(3, 400), (600, 1040), (2, 40016)])
def test_rmsnorm_fp8_far_products(nv, m, k, h_exp, g_exp):
    """The codes are those of the exact products, whatever range they are in."""
    eps = 2.0 ** -126
    h = WL.bf16_bits_from_f32(WL.f32_from_bf16_bits(WL.normal_bf16((m, k), 1.0, 310 + k)) * np.float32(2.0 ** h_exp))
    g = WL.bf16_bits_from_f32(WL.f32_from_bf16_bits(WL.normal_bf16((k,), 1.0, 311 + k)) * np.float32(2.0 ** g_exp))
    h[-1, 128:256] = 0                       # a block of zeros, and one with an ordinary product
    g[:4] = WL.bf16_bits_from_f32(np.float32([2.0 ** (60 if g_exp < 0 else -60)] * 4))
    codes, scales, _ = nv.rmsnorm_fp8(bf16(h), bf16(g), eps)
    rc, rs = F.norm(f64(h), f64(g), eps)
    assert np.array_equal(host(codes), rc)
    # rs, and its rounding where it is subnormal: the largest value's (then divided by 448) and its own.
    assert np.all(np.abs(host(scales) - rs) <= norm_tolerance(k) * rs + 1.01 * 2.0 ** -150)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1024, 40960])
def test_rmsnorm_fp8_value_not_finite(nv, k):
    """A value that overflows though its product does not: scale NaN and codes 0x7F in its block alone."""
    x, g = np.zeros((2, k), dtype=np.float32), np.ones(k, dtype=np.float32)
    x[:, 200], g[200], x[1, 600] = 1.0, 3e38, 1.0
    codes, scales, _ = nv.rmsnorm_fp8(*(bf16(WL.bf16_bits_from_f32(a)) for a in (x, g)), EPS)
    codes, scales = host(codes), host(scales)
    nan = np.zeros(scales.shape, dtype=bool)
    nan[:, 1] = True
    assert np.array_equal(np.isnan(scales), nan) and np.all(codes[:, 128:256] == 0x7F)
    assert codes[1, 600] == 0x7E and not np.delete(codes, [*range(128, 256), 600], axis=1).any()


def silu_check(codes, scales, v):
    """Codes and scales of v (float64) when v is computed in FP32 within delta: log2(e) g is carried in two floats and
    the hardware's exp2 is within 1 ulp, so exp has about 4 u; the sum, division and product add u each, and the
    quotient against an amax with the same error doubles that: 16 u is twice what they add up to."""
    delta = 16 * U
    amax = F.block_amax(v, 1)
    assert np.all(np.abs(scales - amax / 448) <= delta * amax / 448 + 2.0 ** -149)
    q = np.abs(F.quotients(v, 1))
    got = F.values(codes)
    step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)
    assert np.all(np.abs(np.abs(got) - q) <= step / 2 + delta * q)
    assert np.all((got == 0) | (np.sign(got) == np.sign(v)))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(1, 16), (5, 128), (7, 400), (8, 17408), (600, 8192), (3, 20000)])
def test_silu_mul_fp8(nv, m, n):
    b = WL.normal_bf16((m, 2 * n), 3.0, 400 + n)
    codes, scales = nv.silu_mul_fp8(bf16(b))
    silu_check(host(codes), host(scales), F.silu_mul(f64(b[:, :n]), f64(b[:, n:])))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", MANY_BLOCKS)
def test_silu_mul_fp8_many_blocks(nv, m, n):
    test_silu_mul_fp8(nv, m, n)


@pytest.mark.gpu
def test_silu_mul_fp8_extremes(nv):
    """Gates from -3e38 to 3e38, with blocks apart so that small values keep their own scale; not finite blocks."""
    gates = np.float32([-3e38, -200, -104, -90, -87, -60, -20, -1, -1e-3, -1e-30, 0, 1e-30, 1e-3, 1, 20, 87, 90, 3e38])
    b = np.zeros((gates.size, 2 * 128), dtype=np.float32)
    b[:, :128] = gates[:, None] * np.linspace(0.5, 1, 128)[None]
    b[:, 128:] = np.where(np.abs(gates)[:, None] > 1e6, 0.25, 1.5)
    bits = WL.bf16_bits_from_f32(b)
    codes, scales = nv.silu_mul_fp8(bf16(bits))
    v = F.silu_mul(f64(bits[:, :128]), f64(bits[:, 128:]))
    keep = np.abs(v).max(axis=1) == 0
    keep |= np.abs(v).max(axis=1) > 2.0 ** -120       # results below FP32's normal range lose their last bits
    silu_check(host(codes)[keep], host(scales)[keep], v[keep])
    for bad in (np.inf, -np.inf, np.nan):
        for col in (3, 128 + 3):
            c = b[13:15].copy()
            c[0, col] = bad
            codes, scales = nv.silu_mul_fp8(bf16(WL.bf16_bits_from_f32(c)))
            assert np.all(host(codes)[0] == 0x7F) and np.isnan(host(scales)[0]).all()
            assert np.isfinite(host(scales)[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [400, 5120, 40000])
def test_silu_mul_fp8_far_gates(nv, n):
    """silu(gate) far below FP32's normal range, or a subnormal gate's half, times an up that brings it back: blocks
    whose gates have one size each, the ups another, so that every block's results are normal FP32 numbers."""
    gates = np.float32([-86, -87.5, -88, -95, -104, -120, -150, -170, 2.0 ** -130, -2.0 ** -128, 2.0 ** -120, -64, -30, -3])
    ups = np.float32([1, 1, 2, 64, 1e8, 1e20, 1e37, 3e38, 1e30, 1e20, 1e10, 1e-5, 1e38, 1e38])
    rng = np.random.default_rng(410 + n)
    b = np.empty((gates.size, 2 * n), dtype=np.float32)
    b[:, :n] = gates[:, None] * rng.uniform(0.97, 1, (1, n))
    b[:, n:] = ups[:, None] * rng.uniform(0.01, 1, (1, n)) * rng.choice([-1, 1], (1, n))
    bits = WL.bf16_bits_from_f32(b)
    codes, scales = nv.silu_mul_fp8(bf16(bits))
    v = F.silu_mul(f64(bits[:, :n]), f64(bits[:, n:]))
    amax = F.block_amax(v, 1)
    assert 2.0 ** -122 < amax.min() and np.abs(v).max() < 2.0 ** 127
    # As silu_check, with the FP32 rounding of a subnormal value (2^-150) on top.
    delta, scales = 16 * U, host(scales)
    assert np.all(np.abs(scales - amax / 448) <= delta * amax / 448 + 2.0 ** -149)
    q, got = np.abs(F.quotients(v, 1)), F.values(host(codes))
    step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)
    low = 448 * 2.0 ** -150 / F.spread(amax, 1, *v.shape)
    assert np.all(np.abs(np.abs(got) - q) <= step / 2 + delta * q + low)
    assert np.all((got == 0) | (np.sign(got) == np.sign(v)))


# More blocks and rows than one dimension of a launch holds, and offsets that pass 32 bits: the same as call by call on
# parts (every block stands for itself).
@pytest.mark.gpu
def test_fp8_quantize_more_blocks_than_a_launch(nv):
    part = bf16(WL.normal_bf16((4096, 16), 1.0, 420))
    codes, scales = nv.fp8_quantize(part)
    reps, rest = 2 ** 16, 37                                   # 2^28 rows of one block, and a few
    x = torch.cat([part.repeat(reps, 1), part[:rest]])
    got, got_scales = nv.fp8_quantize(x)
    del x
    assert bool((got[:4096 * reps].view(reps, 4096, 16) == codes).all()) and torch.equal(got[4096 * reps:], codes[:rest])
    assert bool((got_scales[:4096 * reps].view(reps, 4096, 1) == scales).all())
    assert torch.equal(got_scales[4096 * reps:], scales[:rest])


@pytest.mark.gpu
def test_fp8_producers_rows_of_2_to_the_28(nv):
    """Rows whose offsets do not fit the 32 bits of the form for shorter ones."""
    rows, k, part = 2, 2 ** 28 + 2 ** 16, 2 ** 16
    torch.manual_seed(421)
    x = torch.randn((rows, k), device="cuda", dtype=torch.bfloat16)
    for block_rows in (1, 128):
        codes, scales = nv.fp8_quantize(x, block_rows)
        for j in range(0, k, 64 * part):
            piece = x[:, j:j + 64 * part].contiguous()
            want, want_scales = nv.fp8_quantize(piece, block_rows)
            assert torch.equal(codes[:, j:j + 64 * part], want)
            assert torch.equal(scales[:, j // 128:(j + 64 * part) // 128], want_scales)
    up = torch.randn((rows, k), device="cuda", dtype=torch.bfloat16)
    codes, scales = nv.silu_mul_fp8(torch.cat([x, up], 1))
    want, want_scales = nv.silu_mul_fp8(torch.cat([x.view(-1, part), up.view(-1, part)], 1))
    assert torch.equal(codes.view(-1, part), want) and torch.equal(scales.view(-1, part // 128), want_scales)


@pytest.mark.gpu
def test_fp8_producers_more_rows_than_a_launch_dimension(nv):
    m, k = 2 ** 20 + 37, 16
    xb, gb = WL.normal_bf16((m, k), 1.0, 422), WL.normal_bf16((k,), 1.0, 423)
    x, g = bf16(xb), bf16(gb)
    codes, scales, h = nv.rmsnorm_fp8(x, g, EPS, residual=x)
    for part in (slice(0, m // 2), slice(m // 2, m)):
        for got, want in zip((codes, scales, h), nv.rmsnorm_fp8(x[part], g, EPS, residual=x[part])):
            assert torch.equal(got[part], want)
    codes, scales = nv.fp8_quantize(x.view(m, 1, k), 128)      # one block of 128 x 128 per matrix
    want, want_scales = nv.fp8_quantize(x, 1)
    assert torch.equal(codes.view(m, k), want) and torch.equal(scales.view(m, 1), want_scales)


def operands(m, n, k, seed, e=None):
    """Random operands with uneven scales, as host arrays."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(rng.uniform(-2, 2, (m, 1)))
    lead = () if e is None else (e,)
    w = rng.standard_normal(lead + (n, k)) * 0.02 * np.exp(rng.uniform(-1, 1, lead + (n, 1)))
    return (*F.quantize(x, 1), *F.quantize(w, 128))


def exact_operands(m, n, k, seed, e=None):
    """Operands whose products and sums are exact: codes of 0 and of magnitudes 0.5 .. 3.75 (products of at least
    2^-2 with bits down to 2^-8, none dropped next to one below 2^4), scales 1 and 2.  The sums are multiples of 2^-8,
    and exact in FP32 while their magnitudes stay below 2^16 (checked on sum |x w|, which bounds every
    partial sum in any order).  The output is then the BF16 nearest to the exact sum."""
    rng = np.random.default_rng(seed)
    lead = () if e is None else (e,)

    def codes(shape):
        c = rng.integers(0x30, 0x48, size=shape).astype(np.uint8)      # 0.5 .. 3.75
        return np.where(rng.random(shape) < 0.1, 0, c | (rng.integers(0, 2, size=shape) << 7)).astype(np.uint8)

    def scales(shape):
        return np.exp2(rng.integers(0, 2, size=shape)).astype(np.float32)
    return (codes((m, k)), scales((m, -(-k // 128))), codes(lead + (n, k)),
            scales(lead + (-(-n // 128), -(-k // 128))))


def check_exact(y, ref, bound):
    assert bound.max() < 2.0 ** 16
    want = torch.from_numpy(ref).float().bfloat16().double().numpy()   # exact in FP32, one rounding
    bad = host(y) != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs differ, first {np.argwhere(bad)[:3].tolist()}"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(y, ref, bound, k):
    bad = ~(np.abs(host(y) - ref) <= F.linear_tolerance(ref, bound, k))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs out of tolerance, first {np.argwhere(bad)[:3].tolist()}"


LINEAR_CASES = [(1, 1, 16), (1, 16, 128), (1, 300, 1040), (2, 17, 144), (5, 64, 2048), (15, 130, 400), (16, 128, 512),
                (17, 256, 640), (32, 1000, 1040), (33, 272, 256), (64, 512, 1024), (65, 129, 272), (100, 513, 384),
                (128, 256, 2064), (200, 700, 1936), (256, 256, 128), (257, 300, 4112), (300, 130, 8192),
                (513, 1030, 272), (700, 259, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", LINEAR_CASES)
def test_fp8_linear(nv, m, n, k):
    xq, xs, wq, ws = operands(m, n, k, 500 + m + n + k)
    d = [dev(a) for a in (xq, xs, wq, ws)]
    y = nv.fp8_linear(*d)
    ref, bound = F.linear(xq, xs, wq, ws)
    check(y, ref, bound, k)
    check(nv.fp8_linear(*d, workspace=None), ref, bound, k)
    ex = exact_operands(m, n, k, 501 + m + n + k)
    check_exact(nv.fp8_linear(*(dev(a) for a in ex)), *F.linear(*ex))
    assert torch.equal(nv.fp8_linear(*d), y)                       # the same bits again
    big = torch.full((m + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")   # rows around the output stay
    if n % 8 == 0:
        assert torch.equal(nv.fp8_linear(*d, out=big[1:m + 1]), y)
        assert bool((big[0] == 7).all()) and bool((big[m + 1] == 7).all())


def decoded(codes, scales, block_rows):
    r, k = codes.shape[-2:]
    sp = scales.repeat_interleave(block_rows, -2)[..., :r, :].repeat_interleave(128, -1)[..., :k]
    return codes.view(torch.float8_e4m3fn).float() * sp


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2048, 17408, 640), (4100, 4500, 400), (333, 5000, 4112), (700, 9000, 1040),
                                   (1500, 1030, 2048), (129, 3000, 3088), (8, 17408, 5120), (64, 5120, 4096),
                                   (1, 34816, 5120), (31, 5120, 8208)])
def test_fp8_linear_large_exact(nv, m, n, k):
    """Sizes of every launch plan, with operands whose sums are exact in FP32: equal to torch's FP32 product."""
    d = [dev(a) for a in exact_operands(m, n, k, 650 + m + n + k)]
    x, w = decoded(d[0], d[1], 1), decoded(d[2], d[3], 128)
    assert float((x.abs() @ w.abs().T).max()) < 2.0 ** 16
    want = (x @ w.T).bfloat16()
    for ws in ("auto", None):
        y = nv.fp8_linear(*d, workspace=ws)
        bad = y != want
        assert not bool(bad.any()), f"workspace {ws}: {int(bad.sum())} outputs differ, first {bad.nonzero()[:3].tolist()}"


# Every tile of the GEMM with fewer chunks of K than its ring holds, as many, and more, and with K split.
@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1500, 9000, 128), (4100, 2050, 256), (2048, 9000, 272), (2048, 9000, 384),
                                   (260, 17408, 256), (200, 17408, 384), (260, 9000, 384), (2048, 700, 512),
                                   (130, 17408, 2064), (4100, 260, 2064), (200, 9000, 2064), (4100, 2050, 16),
                                   (200, 17408, 16), (520, 129, 128), (520, 700, 256), (65, 17408, 2064),
                                   (200, 17408, 4112), (100, 8192, 8192), (100, 6144, 8192),
                                   (31, 5003, 8208), (100, 6145, 8192), (64, 5122, 4096)])
def test_fp8_linear_few_chunks_exact(nv, m, n, k):
    d = [dev(a) for a in exact_operands(m, n, k, 750 + m + n + k)]
    x, w = decoded(d[0], d[1], 1), decoded(d[2], d[3], 128)
    assert float((x.abs() @ w.abs().T).max()) < 2.0 ** 16
    y = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.fp8_linear(*d, out=y[:m])
    bad = y[:m] != (x @ w.T).bfloat16()
    assert not bool(bad.any()), f"{int(bad.sum())} outputs differ, first {bad.nonzero()[:3].tolist()}"
    assert bool((y[m] == 7).all())


# More rows, or columns, than one launch dimension holds of the kernels' smallest tiles.
@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1100000, 64, 128), (1048560, 16, 16), (1, 2 ** 26 + 77, 16), (20, 3000000, 16)])
def test_fp8_linear_extreme_sizes_exact(nv, m, n, k):
    torch.manual_seed(800 + m % 100)

    def codes(*shape):
        return torch.randint(0x30, 0x48, shape, device="cuda", dtype=torch.uint8)    # 0.5 .. 3.75, as exact_operands'
    xq, wq = codes(m, k), codes(n, k)
    xs = torch.full((m, 1), 2.0, device="cuda")
    ws = 2.0 ** torch.randint(0, 2, (-(-n // 128), 1), device="cuda").float()
    y = nv.fp8_linear(xq, xs, wq, ws)
    x = xq.view(torch.float8_e4m3fn).float() * 2.0
    for j in range(0, n, 1 << 20):
        w = wq[j:j + (1 << 20)].view(torch.float8_e4m3fn).float()
        w *= ws[j // 128:(j + len(w) + 127) // 128].repeat_interleave(128, 0)[:len(w)]
        bad = y[:, j:j + len(w)] != (x @ w.T).bfloat16()
        assert not bool(bad.any()), f"{int(bad.sum())} outputs differ, first {bad.nonzero()[:3].tolist()}"


# Up to 64 rows: shares of 4, 20, 36, 52 (and 48, 56, 68 in more rounds) rows of W, which cross the blocks of 128 anywhere.
@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 17, 34, 64])
@pytest.mark.parametrize("n,k", [(1000, 272), (5000, 1040), (9003, 272), (13000, 400), (21000, 144), (28001, 256), (34816, 128)])
def test_fp8_linear_shares_exact(nv, m, n, k):
    xq, xs, wq, ws = exact_operands(m, n, k, 900 + m + n + k)
    y = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.fp8_linear(*map(dev, (xq, xs, wq, ws)), out=y[:m])
    ref, bound = (np.concatenate(v, axis=1) for v in zip(*(
        F.linear(xq, xs, wq[i:i + 1024], ws[i // 128:i // 128 + 8]) for i in range(0, n, 1024))))
    check_exact(y[:m], ref, bound)
    assert (y[m] == 7.0).all()


# Scales of X that fit LDS for fewer rows at a time, or not at all.
@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(17, 20, 70000), (60, 9, 33008), (3, 33, 131200), (18, 5, 262160)])
def test_fp8_linear_long_rows(nv, m, n, k):
    xq, xs, wq, ws = operands(m, n, k, 950 + m)
    y = nv.fp8_linear(*map(dev, (xq, xs, wq, ws)))
    check(y, *F.linear(xq, xs, wq, ws), k)


@pytest.mark.gpu
def test_fp8_linear_takes_float8_tensors(nv):
    xq, xs, wq, ws = (dev(a) for a in operands(3, 40, 144, 600))
    y = nv.fp8_linear(xq.view(torch.float8_e4m3fn), xs, wq.view(torch.float8_e4m3fn), ws)
    assert torch.equal(y, nv.fp8_linear(xq, xs, wq, ws))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40, 300])
def test_fp8_linear_nan_and_zero(nv, m):
    """A NaN code reaches its row or column only, also from the last, short block; zero scales give zeros."""
    n, k = 200, 400
    xq, xs, wq, ws = operands(m, n, k, 700)
    xq[1, k - 1] = 0x7F
    wq[150, 3] = 0xFF
    xs[2] = 0
    y = host(nv.fp8_linear(dev(xq), dev(xs), dev(wq), dev(ws)))
    nan = np.zeros((m, n), dtype=bool)
    nan[1], nan[:, 150] = True, True
    assert np.array_equal(np.isnan(y), nan)
    assert not y[2, np.arange(n) != 150].any()
    clean = operands(m, n, k, 700)
    ref, bound = F.linear(*clean)
    ok = ~nan
    ok[2] = False
    assert np.all(np.abs(y - ref)[ok] <= F.linear_tolerance(ref, bound, k)[ok])


@pytest.mark.gpu
@pytest.mark.parametrize("k", [640, 1040])
@pytest.mark.parametrize("m", [1, 20, 40, 64, 300])
def test_fp8_linear_infinite_scales(nv, m, k):
    """A block's sum times its scale: an infinite scale gives an infinity, not NaN, in its rows or columns alone."""
    n = 300
    xq, wq = torch.full((m, k), 0x38, dtype=torch.uint8), torch.full((n, k), 0x38, dtype=torch.uint8)   # 1.0
    xs, ws = torch.full((m, -(-k // 128)), 0.5), torch.full((3, -(-k // 128)), 2.0)
    want = torch.full((m, n), float(k)).bfloat16()
    ws[1, 4] = math.inf
    want[:, 128:256] = math.inf
    xs[m - 1, 2] = math.inf
    want[m - 1] = math.inf
    args = [a.cuda() for a in (xq, xs, wq, ws)]
    assert torch.equal(nv.fp8_linear(*args).cpu(), want)
    route = torch.zeros((m, 1), dtype=torch.int32, device="cuda")
    assert torch.equal(nv.fp8_linear_grouped(*args[:2], route, args[2][None], args[3][None]).cpu()[:, 0], want)


def far_scales(kind, m, n, k, seed, e=None):
    """Operands whose results are normal BF16 numbers although products of two scales are not FP32 numbers, or are
    subnormal ones.  "above": codes of 1 .. 7 steps of 2^-9 (a block's sum is below 2^-5) and products of scales up to
    2.25 2^130; "below": codes 128 .. 448 (a block's sum, all of one sign, is above 2^18) and products of scales from
    2.25 2^-143.  The exponents are split unevenly between the two scales, another way in each block of K.  Every third
    block of K of X is zero, and all from the twelfth on; there the product of the scales is as large as it can be."""
    rng = np.random.default_rng(seed)
    lead, kb, nb = () if e is None else (e,), -(-k // 128), -(-n // 128)
    lo, hi, top = (0x01, 0x08, 130) if kind == "above" else (0x70, 0x7F, -140)
    xq = rng.integers(lo, hi, size=(m, k)).astype(np.uint8)
    wq = rng.integers(lo, hi, size=lead + (n, k)).astype(np.uint8)
    split = rng.integers(5, 120, size=kb) if kind == "above" else rng.integers(-120, -5, size=kb)
    xs = np.exp2(split[None] - rng.integers(0, 2, size=(m, kb))) * rng.choice([1.0, 1.5], size=(m, kb))
    ws = np.exp2(top - split - rng.integers(0, 2, size=lead + (nb, kb))) * rng.choice([1.0, 1.5], size=lead + (nb, kb))
    for b in (b for b in range(kb) if b % 3 == 2 or b >= 12):
        xq[:, 128 * b:128 * (b + 1)] = 0
        xs[:, b], ws[..., b] = 1.5 * 2.0 ** 127, 1.5 * 2.0 ** 127
    return xq, xs.astype(np.float32), wq, ws.astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["above", "below"])
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (3, 300, 1040), (20, 1000, 400), (40, 9003, 272), (64, 5000, 400),
                                   (3, 20, 131200), (100, 513, 384), (200, 5122, 784), (300, 1030, 2064),
                                   (700, 9000, 400), (2048, 2100, 272)])
def test_fp8_linear_far_scales(nv, m, n, k, kind):
    """The scales are applied without forming a product that leaves FP32's range."""
    xq, xs, wq, ws = far_scales(kind, m, n, k, 1200 + m + n + k)
    ref, bound = F.linear(xq, xs, wq, ws)
    assert 2.0 ** -126 < np.abs(ref).min() and np.abs(ref).max() < 2.0 ** 127
    y = nv.fp8_linear(*map(dev, (xq, xs, wq, ws)))
    check(y, ref, bound, k)


# Every tile shape, two launches, slices of K; the last three in which one row in seven has such scales, and the others
# ordinary ones and zeros (of codes and scale) where the far rows have zeros and the largest scales.
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["above", "below"])
@pytest.mark.parametrize("m,n,k,some", [(1500, 9000, 400, False), (4100, 4500, 400, False), (260, 17408, 400, False),
                                        (65, 17408, 2064, False), (200, 9000, 2064, False), (260, 304, 8192, False),
                                        (333, 5000, 4112, True), (1500, 9000, 400, True), (48, 9000, 784, True)])
def test_fp8_linear_far_scales_plans(nv, m, n, k, some, kind):
    xq, xs, wq, ws = far_scales(kind, m, n, k, 1250 + m + n + k)
    if some:
        near = np.arange(m) % 7 != 3
        zero = [b for b in range(xs.shape[1]) if b % 3 == 2 or b >= 12]
        xs[np.ix_(near, zero)] = 0
        xs[near] *= np.float32(2.0 ** (-60 if kind == "above" else 60))
    d = [dev(a) for a in (xq, xs, wq, ws)]
    x, w = (decoded(d[i], d[i + 1].double(), block) for i, block in ((0, 1), (2, 128)))
    ref = x.double() @ w.double().T          # all of one sign: also the sum of magnitudes
    assert 2.0 ** -126 < float(ref.min()) and float(ref.max()) < 2.0 ** 127
    for workspace in ("auto", None):
        y = nv.fp8_linear(*d, workspace=workspace)
        bad = ~((y.double() - ref).abs() <= F.linear_tolerance(1.0, 1.0, k) * ref)
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} out of tolerance, first {bad.nonzero()[:3].tolist()}"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["above", "below"])
@pytest.mark.parametrize("t,topk,e,n,k", [(4, 2, 5, 130, 400), (300, 4, 6, 300, 1040)])
def test_fp8_linear_grouped_far_scales(nv, t, topk, e, n, k, kind):
    xq, xs, wq, ws = far_scales(kind, t, n, k, 1300 + t, e)
    route = routing("uniform", t, topk, e, 1301 + t)
    ref, bound = F.linear_routed(xq, xs, route, wq, ws)
    check(nv.fp8_linear_grouped(*map(dev, (xq, xs, route, wq, ws))), ref, bound, k)


def routing(kind, t, topk, e, seed):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        r = rng.integers(0, e, size=(t, topk))
    elif kind == "skew":
        r = np.minimum(rng.geometric(0.5, size=(t, topk)) - 1, e - 1)
    elif kind == "one":
        r = np.full((t, topk), e - 1)
    else:
        r = np.full((t, topk), -1)
    r = r.astype(np.int32)
    if r.size >= 6 and kind != "none":
        r.flat[2], r.flat[3], r.flat[5] = -1, e, 2 ** 31 - 1
    return r


GROUPED_CASES = [(1, 1, 1, 16, 128, "uniform"), (1, 8, 128, 64, 256, "uniform"), (4, 8, 16, 130, 400, "uniform"),
                 (3, 2, 5, 33, 1040, "none"), (20, 4, 6, 300, 272, "skew"), (130, 2, 3, 64, 512, "one"),
                 (200, 8, 16, 545, 256, "skew"), (300, 4, 6, 300, 1040, "uniform"), (40, 3, 700, 24, 144, "uniform"),
                 (4200, 8, 4, 16, 128, "uniform")]


# Exact sums: without a sort, of one expert more pairs than the 16 of a pass; behind the sort, tiles of 128 pairs with
# few rows, more than half and all of them, ids out of range.
@pytest.mark.gpu
@pytest.mark.parametrize("t,topk,e,n,k,kind", [
    (32, 1, 8, 100, 272, "one"), (64, 1, 8, 259, 400, "skew"), (64, 8, 128, 64, 256, "skew"), (128, 4, 200, 33, 144, "none"),
    (256, 4, 8, 515, 272, "uniform"), (129, 4, 3, 260, 1040, "one"), (700, 2, 9, 1000, 400, "skew"),
    (180, 3, 40, 257, 128, "none"), (2050, 1, 16, 300, 384, "uniform")])
def test_fp8_linear_grouped_exact(nv, t, topk, e, n, k, kind):
    xq, xs, wq, ws = exact_operands(t, n, k, 1000 + t + n + k, e)
    route = routing(kind, t, topk, e, 1100 + t)
    y = torch.full((t + 1, topk, n), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.fp8_linear_grouped(*map(dev, (xq, xs, route, wq, ws)), out=y[:t])
    ref, bound = F.linear_routed(xq, xs, route, wq, ws)
    check_exact(y[:t], ref, bound)
    assert bool((y[t] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("t,topk,e,n,k,kind", GROUPED_CASES)
def test_fp8_linear_grouped(nv, t, topk, e, n, k, kind):
    xq, xs, wq, ws = operands(t, n, k, 800 + t + n + k, e)
    route = routing(kind, t, topk, e, 801)
    d = [dev(a) for a in (xq, xs, route, wq, ws)]
    y = nv.fp8_linear_grouped(*d)
    ref, bound = F.linear_routed(xq, xs, route, wq, ws)
    check(y, ref, bound, k)
    assert not host(y)[(route < 0) | (route >= e)].any()
    ex = exact_operands(t, n, k, 802 + t + n + k, e)
    check_exact(nv.fp8_linear_grouped(dev(ex[0]), dev(ex[1]), d[2], dev(ex[2]), dev(ex[3])),
                *F.linear_routed(ex[0], ex[1], route, ex[2], ex[3]))
    dirty = torch.full((nv.fp8_linear_grouped_workspace_bytes(t, topk, e),), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full_like(y, 3.0)
    assert torch.equal(nv.fp8_linear_grouped(*d, out=out, workspace=dirty), y)


# ---------------------------------------------------------------------------
# The operators together, and how they are called.
# ---------------------------------------------------------------------------
def mlp(nv, x, r, g, gu, down):
    """One MLP block in E4M3: residual + norm -> gate/up -> silu * up -> down; (y, new residual)."""
    q, s, h = nv.rmsnorm_fp8(x, g, EPS, residual=r)
    q, s = nv.silu_mul_fp8(nv.fp8_linear(q, s, *gu))
    return nv.fp8_linear(q, s, *down), h


def close(got, want, tol):
    """Relative 2-norm; the chain's own roundings: E4M3 (2^-4 a value at most) in two operands that both sides round
    alike up to the BF16 rounding between them (2^-8), which moves few codes by a step."""
    got, want = got.double(), want.double()
    assert float((got - want).norm()) <= tol * float(want.norm())


def chain_inputs(m, k, n, seed, e=None):
    lead = () if e is None else (e,)
    x, r = bf16(WL.normal_bf16((m, k), 1.0, seed)), bf16(WL.normal_bf16((m, k), 2.0, seed + 1))
    g = bf16(WL.normal_bf16((k,), 1.0, seed + 2))
    gu, down = bf16(WL.normal_bf16(lead + (2 * n, k), 0.05, seed + 3)), bf16(WL.normal_bf16(lead + (k, n), 0.05, seed + 4))
    return x, r, g, gu, down


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n", [(1, 512, 384), (7, 1040, 400), (150, 512, 1024), (300, 2048, 1040)])
def test_fp8_mlp_block(nv, m, k, n):
    """The operators in a row against the same steps in float64, with the operands rounded to E4M3 by the oracle's
    definition and BF16 between the steps."""
    x, r, g, gu, down = chain_inputs(m, k, n, 900 + m)
    guq, dq = nv.fp8_quantize(gu, 128), nv.fp8_quantize(down, 128)
    y, h = mlp(nv, x, r, g, guq, dq)
    hd = host((x.float() + r.float()).bfloat16())
    assert np.array_equal(host(h), hd)
    cq, cs = F.norm(hd, host(g), EPS)
    a, _ = F.linear(cq, cs, *F.quantize(host(gu), 128))
    a = torch.from_numpy(a).bfloat16().double().numpy()
    q, s = F.quantize(F.silu_mul(a[:, :n], a[:, n:]), 1)
    want, _ = F.linear(q, s, *F.quantize(host(down), 128))
    # gate/up outputs: 2^-8 rounding on both sides and the products' 7 2^-13 of sum |x w|; at most a code step (2^-3)
    # where they move a value over a border, which a share of about 2^-8 / 2^-4 of the values is near to.
    close(y.cpu(), torch.from_numpy(want), 2.0 ** -8 + 2.0 ** -3 * (2.0 ** -4) ** 0.5)


@pytest.mark.gpu
def test_fp8_moe_block(nv):
    """norm -> grouped gate/up -> silu * up -> grouped down (one row per pair), with padding tokens: row for row the
    same bits as the dense operators on each expert's rows."""
    t, topk, e, k, n = 37, 2, 5, 512, 272
    x, r, g, gu, down = chain_inputs(t, k, n, 950, e)
    guq, dq = nv.fp8_quantize(gu, 128), nv.fp8_quantize(down, 128)
    route = routing("uniform", t, topk, e, 951)
    route[30:] = -1
    rd = dev(route)
    q, s, h = nv.rmsnorm_fp8(x, g, EPS, residual=r)
    a = nv.fp8_linear_grouped(q, s, rd, *guq)
    q2, s2 = nv.silu_mul_fp8(a.view(t * topk, 2 * n))
    y = nv.fp8_linear_grouped(q2, s2, rd.view(t * topk, 1), *dq).view(t, topk, k)
    valid = (route >= 0) & (route < e)
    assert not host(y)[~valid].any() and not host(a)[~valid].any()
    ra, ba = F.linear_routed(host(q), host(s), route, host(guq[0]), host(guq[1]))
    check(a, ra, ba, k)
    ry, by = F.linear_routed(host(q2), host(s2), route.reshape(-1, 1), host(dq[0]), host(dq[1]))
    check(y, ry.reshape(t, topk, k), by.reshape(t, topk, k), n)


@pytest.mark.gpu
def test_fp8_graph_replays_match_eager(nv):
    """A whole MLP and MoE step captured once and replayed with other work in between, on new inputs too; two graphs
    captured on one stream keep apart."""
    x, r, g, gu, down = chain_inputs(260, 512, 1024, 970)
    guq, dq = nv.fp8_quantize(gu, 128), nv.fp8_quantize(down, 128)
    stack = nv.fp8_quantize(bf16(WL.normal_bf16((6, 272, 512), 0.05, 975)), 128)
    routes = [dev(routing("skew", 260, 4, 6, 976)), dev(routing("uniform", 3, 2, 6, 977))]
    long_w = nv.fp8_quantize(bf16(WL.normal_bf16((304, 8192), 0.05, 978)), 128)
    long_x = nv.fp8_quantize(bf16(WL.normal_bf16((260, 8192), 1.0, 979)))
    assert nv.fp8_linear_workspace_bytes(260, 304, 8192) > 0      # K split: two launches and a workspace

    def step():
        q, s, h = nv.rmsnorm_fp8(x, g, EPS, residual=r)
        y, _ = mlp(nv, x, r, g, guq, dq)
        few = nv.fp8_linear_grouped(q[:3].contiguous(), s[:3].contiguous(), routes[1], *stack)
        return [h, y, nv.fp8_linear_grouped(q, s, routes[0], *stack), few, nv.fp8_linear(*long_x, *long_w),
                nv.fp8_linear(q[:5].contiguous(), s[:5].contiguous(), *guq), *nv.fp8_quantize(x, 128)]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            out = step()
        graphs.append((gr, out))
    torch.cuda.synchronize()
    for rep in range(3):
        x.copy_(bf16(WL.normal_bf16((260, 512), 1.0, 980 + rep)))
        want = step()
        torch.cuda.synchronize()
        for gr, out in graphs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for gr, _ in graphs:
            gr.replay()
        step()                                                     # eager work beside the replays
        torch.cuda.synchronize()
        for i, (_, out) in enumerate(graphs):
            for j, (o, ref) in enumerate(zip(out, want)):
                assert torch.equal(o.view(torch.uint8), ref.view(torch.uint8)), (rep, i, j)


@pytest.mark.gpu
def test_fp8_two_streams_at_once(nv):
    """Calls in flight on two streams, each with its own workspace, give the results of one after the other."""
    w = [nv.fp8_quantize(bf16(WL.normal_bf16((304, 8192), 0.05, 990 + i)), 128) for i in range(2)]
    x = [nv.fp8_quantize(bf16(WL.normal_bf16((260, 8192), 1.0, 992 + i))) for i in range(2)]
    want = [nv.fp8_linear(*x[i], *w[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(nv.fp8_linear(*x[i], *w[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.gpu
def test_fp8_binding_refusals(nv):
    x = bf16(WL.normal_bf16((4, 256), 1.0, 1000))
    g = bf16(WL.normal_bf16((256,), 1.0, 1001))
    q, s = nv.fp8_quantize(x)
    wq, ws = nv.fp8_quantize(bf16(WL.normal_bf16((64, 256), 1.0, 1002)), 128)
    route = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    bad = [
        lambda: nv.fp8_quantize(x.float()), lambda: nv.fp8_quantize(x.cpu()), lambda: nv.fp8_quantize(x[:, ::2]),
        lambda: nv.fp8_quantize(x[0]), lambda: nv.fp8_quantize(x, 64), lambda: nv.fp8_quantize(x[:, :8].contiguous()),
        lambda: nv.rmsnorm_fp8(x, g[:128].contiguous()), lambda: nv.rmsnorm_fp8(x, g, residual_out=x),
        lambda: nv.rmsnorm_fp8(x, g, residual=x[:2]), lambda: nv.rmsnorm_fp8(x, g.float()),
        lambda: nv.silu_mul_fp8(x[0]), lambda: nv.silu_mul_fp8(x[:, :255].contiguous()),
        lambda: nv.silu_mul_fp8(x[:, :16].contiguous()),
        lambda: nv.fp8_linear(q, s[:2].contiguous(), wq, ws), lambda: nv.fp8_linear(q.int(), s, wq, ws),
        lambda: nv.fp8_linear(q, s, wq[:, :128].contiguous(), ws), lambda: nv.fp8_linear(q, s, wq, ws.double()),
        lambda: nv.fp8_linear(q, s, wq, ws, out=x), lambda: nv.fp8_linear(q, s, wq, ws, workspace="none"),
        lambda: nv.fp8_linear(q, s, wq.cpu(), ws),
        lambda: nv.fp8_linear_grouped(q, s, route, wq, ws), lambda: nv.fp8_linear_grouped(q, s, route[:2], wq[None], ws[None]),
        lambda: nv.fp8_linear_grouped(q, s, route.long(), wq[None], ws[None]),
        lambda: nv.fp8_linear_grouped(q, s, route[:, :0], wq[None], ws[None]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(nv.NVFP4Error):
        nv.rmsnorm_fp8(x, g, 0.0)
    with pytest.raises(nv.NVFP4Error):
        nv.rmsnorm_fp8(x, g, residual=x, residual_out=x)           # over the input
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_linear_grouped(q, s, route, wq[None].contiguous(), ws[None].contiguous(), workspace=small)
    # empty batches
    assert nv.fp8_quantize(x[:0])[0].shape == (0, 256) and nv.silu_mul_fp8(x[:0])[1].shape == (0, 1)
    assert nv.rmsnorm_fp8(x[:0], g, residual=x[:0])[2].shape == (0, 256)
    assert nv.fp8_linear(q[:0], s[:0], wq, ws).shape == (0, 64)
    assert nv.fp8_linear_grouped(q[:0], s[:0], route[:0], wq[None], ws[None]).shape == (0, 2, 64)


def test_fp8_binding_refuses_mixed_devices():
    class On:
        def __init__(self, device):
            self.device = torch.device(device)
    assert B._one_device(On("cuda:1"), None, On("cuda:1")) == torch.device("cuda:1")
    with pytest.raises(ValueError, match="different devices"):
        B._one_device(On("cuda:0"), On("cuda:1"))


def test_fp8_binding_runs_on_the_tensors_device(monkeypatch):
    """A call whose tensors are on another device than the current one switches to it and takes its stream."""
    seen = []
    now = {"dev": 0}

    class Guard:
        def __init__(self, device):
            self.to = device.index

        def __enter__(self):
            self.before, now["dev"] = now["dev"], self.to

        def __exit__(self, *a):
            now["dev"] = self.before
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["dev"])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(B, "_stream_of", lambda d: 100 + d.index)
    for index in (0, 1):
        B._call(lambda *a: seen.append((now["dev"], a)) or 0, "f", torch.device("cuda", index), 7)
    assert seen == [(0, (7, 100)), (1, (7, 101))] and now["dev"] == 0
