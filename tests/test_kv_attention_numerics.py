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
