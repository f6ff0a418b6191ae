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


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows, g, d", [(40, 8, 128), (40, 8, 256), (12, 4, 64)], ids=["many", "many256", "few"])
def test_captured_with_other_lengths(nv, rows, g, d, fmt):  # noqa: F811
    """Two graphs that share a workspace, replayed in turn with lengths and chunks that change in between: rows move from
    one sequence to another and some belong to none."""
    rng = np.random.default_rng(730)
    table = i32(rng.permutation(96).reshape(3, 32))
    cache = device_cache(nv, fmt, make_cache(rng, fmt, 96, 16, 2, d))
    q = [rand(rng, (rows, 2 * g, d), torch.bfloat16) for _ in range(2)]
    lens, start = i32([100, 200, 300]), i32([0, 3, 4, rows])
    ws = torch.empty(nv.kv_attention_workspace_bytes(2, d, 2 * g, rows, 3), dtype=torch.uint8, device="cuda")
    out = [torch.zeros_like(x) for x in q]

    def call(i, out):
        return nv.kv_attention(q[i], cache, table, lens, start, window=150, out=out, workspace=ws)
    for i in range(2):
        call(i, out[i])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i, out[i])
    for lens_now, start_now in (([100, 200, 300], [0, 3, 4, rows]), ([512, 1, 40], [0, rows - 2, rows - 1, rows]),
                                ([7, 0, 511], [2, 5, 5, rows - 4]), ([90, 500, 8], [0, 0, rows - 1, rows - 1])):
        lens.copy_(i32(lens_now))
        start.copy_(i32(start_now))
        for x in q:
            x.copy_(rand(rng, x.shape, x.dtype))
        for x in out:
            x.fill_(5.0)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], call(i, torch.full_like(q[i], 5.0)))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_heads_outside_rows_and_shared_by_rows(nv, fmt):  # noqa: F811
    """Keys with heads outside rows, one value head for all, queries with heads outside rows: strides that are allowed."""
    rng = np.random.default_rng(740)
    heads, g, d = 3, 5, 96
    for lens, n in (([60, 33], [1, 1]), ([200, 77], [50, 20])):
        nb, table, lens, start = make_batch(rng, lens, n, 24)
        c = make_cache(rng, fmt, nb, 24, heads, d)
        cache = device_cache(nv, fmt, c)
        rows = int(start[-1])
        k = rand(rng, (heads, rows, d), torch.bfloat16).transpose(0, 1)
        v = rand(rng, (rows, 1, d), torch.bfloat16).expand(rows, heads, d)
        nv.kv_append(k, v, cache, i32(table), i32(lens), i32(start))
        c = test_kv_ops.K.append(fmt, c, test_kv_ops.f64(k), test_kv_ops.f64(v), table, lens, start)
        test_kv_ops.same_cache(test_kv_ops.host_cache(cache, c), c)
        q = rand(rng, (heads * g, rows, d), torch.float16).transpose(0, 1)
        got = nv.kv_attention(q, cache, i32(table), i32(lens), i32(start))
        within(got, q, c, fmt, table, lens, start, d ** -0.5, 0, 2.0 ** -22 if fmt == "nvfp4" else 2.0 ** -16)
