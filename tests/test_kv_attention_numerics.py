"""Numbers at the edges of attention over the paged FP4 cache: HIP kernels against the float64 oracle (GPU), in the
kernel for few rows a sequence and in the one for many."""
import numpy as np
import pytest
import torch

from oracle import kv_ops_oracle as K
from test_kv_ops import HALF_STEP, TINY, TYPES, device_cache, f64, i32, make_batch, make_cache, rand


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_weight_only_amd as nv
    nv.lib()
    return nv


def within(got, q, c, fmt, table, lens, start, scale, window, weight):
    """The oracle's bound (R28) with weights rounded by `weight`, half a step of the output's type on top."""
    y, bound, mine = K.attention(fmt, c, f64(q), table, lens, start, scale, window, weight)
    off = np.abs(f64(got) - y) - (bound + HALF_STEP[q.dtype] * (np.abs(y) + bound) + TINY[q.dtype])
    assert np.isfinite(y).all() and np.isfinite(f64(got)).all()
    assert (off[mine] <= 0).all(), f"{off.max()} over, worst at {np.unravel_index(np.argmax(off), off.shape)}"


FEW, MANY = (1, 4), (3, 16)  # rows and query heads of a key/value head: 4 and 48 packed rows a sequence


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_weights_have_more_bits_than_the_output(nv, shape, dt, fmt):
    """A few tokens whose values nearly cancel, so that the output's own rounding is small next to its terms, and small
    scores, so that the FP32 sums' part of the bound is: what is left shows the weights' rounding.  Two FP16 terms round
    by 2^-22 and two BF16 ones by 2^-16 (one by 2^-11 and 2^-8); NVFP4 with BF16 outputs has one for many rows."""
    per, g = shape
    if per > 1 and fmt == "nvfp4" and dt == "bf16":
        weight = 2.0 ** -11
    else:
        weight = 2.0 ** -22 if fmt == "nvfp4" else 2.0 ** -16
    dt, rng = TYPES[dt], np.random.default_rng(500)
    lens = rng.integers(per + 1, per + 5, size=64).tolist()
    nb, table, lens, start = make_batch(rng, lens, [per] * 64, 16)
    c = make_cache(rng, fmt, nb, 16, 1, 64)
    cache = device_cache(nv, fmt, c)
    q = rand(rng, (64 * per, g, 64), dt)
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=0.02)
    within(got, q, c, fmt, table, lens, start, 0.02, 0, weight)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("fmt, size, kt, scale", [
    ("nvfp4", 2.0 ** -130, 2.0 ** -24, 0.125),         # scores of nearly 0: the mean of the values that a row sees
    ("nvfp4", 2.0 ** -130, 2.0 ** 30, 2.0 ** 100),     # the scales' product above FP32's range, scores of ordinary size
    ("nvfp4", 2.0 ** 125, 2.0 ** -120, 2.0 ** -5),
    ("nvfp4", 2.0 ** 100, 2.0 ** -60, -2.0 ** -100),   # the scales' product below FP32's range
    ("mxfp4", 2.0 ** -128, None, 3e38),                # times log2 e above FP32's range
    ("mxfp4", 2.0 ** -130, None, 0.125),
    ("mxfp4", 2.0 ** 125, None, 2.0 ** -125),
])
def test_far_queries_and_scales(nv, fmt, size, kt, scale, shape):
    """Queries near BF16's ends with scales that bring the scores back, where every row has tokens that it does not see."""
    per, g = shape
    rng = np.random.default_rng(501)
    lens = rng.integers(per + 1, 90, size=5).tolist()
    nb, table, lens, start = make_batch(rng, lens, [per] * 5, 16)
    c = make_cache(rng, fmt, nb, 16, 2, 64)
    if kt is not None:
        c["k_tscale"] = np.float32(kt)
    cache = device_cache(nv, fmt, c)
    q = torch.from_numpy(np.clip(rng.normal(0, size, size=(5 * per, 2 * g, 64)), -3e38, 3e38)).to(torch.bfloat16).cuda()
    for window in (None, 7):
        got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale, window=window)
        within(got, q, c, fmt, table, lens, start, scale, window or 0, 2.0 ** -11)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_infinite_queries(nv, shape, dt, fmt):
    """An infinity in a query makes every score one, with positive keys of one sign: the softmax is NaN for -inf as for
    inf, unless the row sees nothing.  The other rows are as they are without it."""
    per, g = shape
    dt, rng = TYPES[dt], np.random.default_rng(502)
    lens = [1, 40, 90, 0, 400]
    nb, table, lens, start = make_batch(rng, lens, [per] * 5, 16)
    c = make_cache(rng, fmt, nb, 16, 1, 64)
    c["k_codes"] = rng.integers(1, 8, size=c["k_codes"].shape, dtype=np.uint8) * np.uint8(17)
    cache = device_cache(nv, fmt, c)
    q = rand(rng, (5 * per, g, 64), dt)
    clean = f64(nv.kv_attention(q, cache, i32(table), i32(lens), i32(start)))
    sees = np.array([int(n) - per + i >= 0 for n in lens for i in range(per)])
    for value in (float("-inf"), float("inf")):
        x = q.clone()
        x[:, 1, 9] = value
        got = f64(nv.kv_attention(x, cache, i32(table), i32(lens), i32(start)))
        assert np.isnan(got[sees, 1]).all() and (got[~sees, 1] == 0).all()
        others = [0, *range(2, g)]
        assert np.array_equal(got[:, others], clean[:, others])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_tiny_value_scales(nv, shape):
    """A value tensor scale whose quotient by the sum of many weights is below FP32's range, while the outputs are not:
    sequences within a workgroup's share, and one that is joined."""
    per, g = shape
    rng = np.random.default_rng(503)
    lens = [600] * 150 + [30000]
    nb, table, lens, start = make_batch(rng, lens, [per] * 151, 64)
    c = make_cache(rng, "nvfp4", nb, 64, 1, 64)
    c["v_codes"] = rng.integers(1, 8, size=c["v_codes"].shape, dtype=np.uint8) * np.uint8(17)
    c["v_scales"][:] = 0x60
    c["v_tscale"] = np.float32(2.0 ** -130)
    cache = device_cache(nv, "nvfp4", c)
    q = rand(rng, (151 * per, g, 64), torch.bfloat16)
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=0.001)
    within(got, q, c, "nvfp4", table, lens, start, 0.001, 0, 2.0 ** -11)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_sums_of_large_mxfp4_values(nv, shape):
    """500 tokens of 6 * 2^116, n |v| = 2^127.55, the first of them with a score just below the step at which the maximum
    is taken again, so that the others' weights are the largest that there are."""
    per, g = shape
    rng = np.random.default_rng(504)
    n = 500
    nb, table, lens, start = make_batch(rng, [n, n], [per, per], 16)
    c = make_cache(rng, "mxfp4", nb, 16, 1, 64)
    c["k_codes"][:], c["k_scales"][:] = 0x22, 127                 # 1.0
    c["v_scales"][:] = 243
    c["v_codes"] = np.broadcast_to(rng.choice(np.array([0x77, 0xFF], np.uint8), size=(1, 1, 1, 32)), c["v_codes"].shape).copy()
    for s in range(2):
        for t in range(32):
            c["k_codes"][table[s, t // 16], t % 16] = 0
    cache = device_cache(nv, "mxfp4", c)
    q = torch.ones((2 * per, g, 64), dtype=torch.bfloat16, device="cuda")
    scale = 7.9 * np.log(2) / 64
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale)
    within(got, q, c, "mxfp4", table, lens, start, np.float64(np.float32(scale)), 0, 2.0 ** -16)
    assert (f64(got) == K.values("mxfp4", c["v_codes"][table[0, 0], 0], c["v_scales"][table[0, 0], 0])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [FEW, MANY, (9, 16)], ids=["few", "many", "more"])
def test_widest_windows(nv, shape):
    """Windows up to 2^31 - 1 (and beyond, which the binding takes as that), rows before token 0 among those that they
    let see; lengths far behind the table, whose rows see its end through a long window and nothing through a short one."""
    per, g = shape
    rng = np.random.default_rng(505)
    lens = [per - 1 if per > 1 else 0, 3, 40, 200]
    nb, table, lens, start = make_batch(rng, lens, [per] * 4, 16)
    c = make_cache(rng, "nvfp4", nb, 16, 1, 64)
    cache = device_cache(nv, "nvfp4", c)
    q = rand(rng, (4 * per, g, 64), torch.bfloat16)
    plain = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start))
    within(plain, q, c, "nvfp4", table, lens, start, 0.125, 0, 2.0 ** -11)
    for window in (2 ** 30, 2 ** 31 - 5, 2 ** 31 - 1, 2 ** 40, 2 ** 70):
        assert torch.equal(nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=window), plain)
    far = np.array([2 ** 31 - 1, 2 ** 31 - 40, 10 ** 6, 300], np.int64)
    for window in (7, 100, 2 ** 31 - 1):
        got = nv.kv_attention(q, cache, i32(table), i32(far), i32(start), window=window)
        within(got, q, c, "nvfp4", table, far, start, 0.125, window, 2.0 ** -11)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_scores_beyond_2_to_the_24(nv, shape, sign, fmt):
    """Scores of 2^23 to 2^29, where FP32's step is 1 to 64: later tokens lie a little above the first ones' maximum, and
    the weights' offset from it is rounded.  All values are the same, so that every mean of them is."""
    per, g = shape
    rng = np.random.default_rng(506)
    n, seqs = 1000, 200
    nb, table, lens, start = make_batch(rng, [n], [per], 16)
    lens, start = np.repeat(lens, seqs), np.arange(seqs + 1, dtype=np.int32) * per
    table = np.repeat(table, seqs, 0)
    c = make_cache(rng, fmt, nb, 16, 1, 64)
    c["k_codes"][:], c["k_scales"][:] = 0, 0x38 if fmt == "nvfp4" else 127
    c["k_codes"][..., :16] = 0x77                      # 32 elements of 6 times 2^8
    c["k_scales"][..., :32 // K.GROUP[fmt]] = 0x78 if fmt == "nvfp4" else 135
    last = -32 // K.GROUP[fmt]
    c["k_scales"][..., last:] = 0x10 if fmt == "nvfp4" else 122  # steps of 2^-6
    for t in range(n):
        c["k_codes"][table[0, t // 16], t % 16, 0, 16:] = 0 if t < 32 else rng.integers(0, 8, size=16)
    c["k_tscale"] = c["v_tscale"] = np.float32(1.0) if fmt == "nvfp4" else None
    c["v_codes"][:], c["v_scales"][:] = np.tile(np.array([0x22, 0x4A], np.uint8), 16), 0x38 if fmt == "nvfp4" else 127
    cache = device_cache(nv, fmt, c)
    want = K.values(fmt, c["v_codes"][0, 0], c["v_scales"][0, 0], c["v_tscale"])
    q = torch.full((seqs * per, g, 64), float(sign), dtype=torch.bfloat16, device="cuda")
    for power in np.linspace(23, 29, 25):
        scale = 2.0 ** power / (32 * 1536) / np.log2(np.e)
        got = f64(nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale))
        wrong = got != want
        assert not wrong.any(), f"2^{power}: {int(wrong.sum())} wrong, the first of them {got[wrong][:3]}"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_small_elements_and_small_weights_count(nv, shape, dt, fmt):
    """Elements of a query 2^-15 of its largest, which meets zeros in the keys; and 20000 weights of 2^-24 of the largest,
    whose value is 0: subnormal numbers of FP16 on the matrix cores."""
    per, g = shape
    dt, rng = TYPES[dt], np.random.default_rng(507)
    weight = 2.0 ** -16 if fmt == "mxfp4" else 2.0 ** -11
    nb, table, lens, start = make_batch(rng, [70, 200], [per, per], 16)
    c = make_cache(rng, fmt, nb, 16, 1, 64)
    c["k_codes"][..., 0] &= 0xF0                       # element 0
    cache = device_cache(nv, fmt, c)
    q = rand(rng, (2 * per, g, 64), dt, 2.0 ** -13)
    q[..., 0] = 4.0
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=2.0 ** 9)
    within(got, q, c, fmt, table, lens, start, 2.0 ** 9, 0, weight)
    n = 20000
    nb, table, lens, start = make_batch(rng, [n], [per], 64)
    c = make_cache(rng, fmt, nb, 64, 1, 64)
    c["k_codes"][:], c["k_scales"][:] = 0, 0x38 if fmt == "nvfp4" else 127
    c["v_codes"][:], c["v_scales"][:] = 0x22, 0x38 if fmt == "nvfp4" else 127
    c["k_codes"][table[0, 3], 5] = 0x22                # token 197
    c["v_codes"][table[0, 3], 5] = 0
    c["k_tscale"] = c["v_tscale"] = np.float32(1.0) if fmt == "nvfp4" else None
    cache = device_cache(nv, fmt, c)
    q = torch.ones((per, g, 64), dtype=dt, device="cuda")
    scale = 24 * np.log(2) / 64
    got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale)
    within(got, q, c, fmt, table, lens, start, np.float64(np.float32(scale)), 0, weight)
    assert (np.abs(f64(got) / (n * 2.0 ** -24) - 1) < 0.1).all()
