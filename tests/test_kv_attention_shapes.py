"""Attention over the paged FP4 cache in the kernel that takes 32 rows at a time (17 to 32 packed rows a sequence on
average, heads of up to 128), and its joins: HIP kernels against the float64 oracle (GPU)."""
import numpy as np
import pytest
import torch

import test_kv_ops
from test_kv_attention_numerics import nv, within  # noqa: F401
from test_kv_ops import TYPES, device_cache, i32, make_batch, make_cache, rand

pytestmark = pytest.mark.gpu

# lens, rows, heads, group: packed rows (rows * group) at 16 * seqs + 1, between, and at 32 * seqs; sequences whose tokens
# several workgroups share, and one whose parts are joined by 1024 threads (fewer than 256 outputs' heads, a table of more
# than 2048 tokens).  3 heads leave one of a workgroup's two idle, 4 are two groups of heads.
SHAPES = [
    ([1400], [17], 4, 1),
    ([900, 1300, 333], [8, 8, 8], 4, 4),
    ([900, 1300, 333], [5, 9, 7], 3, 4),
    ([2600], [8], 3, 4),
    ([70, 5000, 31, 900], [16, 16, 16, 16], 1, 2),
    ([3000], [1], 2, 32),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_32_rows(nv, shape, d, dt, fmt):  # noqa: F811
    lens, n, heads, g = SHAPES[shape]
    assert 16 * len(lens) < sum(n) * g <= 32 * len(lens)
    dt, rng = TYPES[dt], np.random.default_rng(700 + shape)
    nb, table, lens, start = make_batch(rng, lens, n, 24)
    c = make_cache(rng, fmt, nb, 24, heads, d)
    cache = device_cache(nv, fmt, c)
    q = rand(rng, (sum(n), heads * g, d), dt)
    weight = 2.0 ** -22 if fmt == "nvfp4" else 2.0 ** -16
    for window in (0, 150):
        got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=window or None)
        within(got, q, c, fmt, table, lens, start, d ** -0.5, window, weight)
        assert torch.equal(got, nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), window=window or None))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_joins_of_few_rows(nv, d, fmt):  # noqa: F811
    """16 rows at a time: the same sequence joined by 1024 threads, by 256 (a table of up to 2048 tokens), and within a
    batch of so many rows that 256 threads join."""
    rng = np.random.default_rng(710)
    for lens, rows, heads, g, extra in (([1900], 1, 8, 5, 1), ([1900], 1, 8, 5, 40), ([2300, 1900], 2, 2, 4, 1),
                                        ([5000] * 8, 8, 8, 4, 1)):
        nb, table, ls, start = make_batch(rng, lens, [1] * rows, 16, extra_blocks=extra)
        c = make_cache(rng, fmt, nb, 16, heads, d)
        cache = device_cache(nv, fmt, c)
        q = rand(rng, (rows, heads * g, d), torch.float16)
        got = nv.kv_attention(q, cache, i32(table), i32(ls))
        within(got, q, c, fmt, table, ls, start, d ** -0.5, 0, 2.0 ** -22 if fmt == "nvfp4" else 2.0 ** -16)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("per", [5, 8])
def test_hidden_values_32_rows(nv, fmt, per):  # noqa: F811
    """NaN blocks and infinities where a wavefront holds two tiles of rows: 4 query heads a key/value head, 5 and 8 rows."""
    test_kv_ops.test_kv_attention_hidden_values(nv, fmt, per)


@pytest.mark.parametrize("shape", [(1, 4), (6, 4), (3, 16)], ids=["few", "few32", "many"])
@pytest.mark.parametrize("dt", list(TYPES))
def test_far_mxfp4_scales(nv, dt, shape):  # noqa: F811
    """Scales of keys and values far apart in MXFP4, FP16 outputs among them (values up to 6 * 2^-1 there)."""
    per, g = shape
    dt, rng = TYPES[dt], np.random.default_rng(720)
    nb, table, lens, start = make_batch(rng, [100, 33, 400], [per] * 3, 16)
    for size in (1e4, 1.0, 1e-4):
        c = make_cache(rng, "mxfp4", nb, 16, 1, 64)
        c["k_scales"] = rng.choice([90, 110, 126, 127], size=c["k_scales"].shape).astype(np.uint8)
        c["v_scales"] = rng.choice([0, 60, 110, 126], size=c["v_scales"].shape).astype(np.uint8)
        cache = device_cache(nv, "mxfp4", c)
        q = rand(rng, (3 * per, g, 64), dt, size)
        scale = float(np.float32(0.125 / size))
        got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start), scale=scale)
        within(got, q, c, "mxfp4", table, lens, start, scale, 0, 2.0 ** -16)
