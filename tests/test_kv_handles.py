"""The handles of a cache and of a rotation (GPU): what the kernels read is what the handle's tensors hold in the call."""
import numpy as np
import pytest
import torch

from oracle import kv_ops_oracle as K
from test_kv_ops import device_cache, i32, make_batch, make_cache, nv, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def test_attributes_are_read_only(nv):  # noqa: F811
    cache = nv.KVCache.zeros(4, 16, 2, 64, "mxfp4")
    rope = nv.Rope(torch.zeros(16, dtype=torch.float64, device="cuda"))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "k_tscale", "v_tscale", "fmt", "device", "num_blocks",
                 "block_size", "heads", "head_dim"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    for name in ("freqs", "amplitude", "interleaved", "rot_dim"):
        with pytest.raises(AttributeError):
            setattr(rope, name, getattr(rope, name))
    assert (cache.num_blocks, cache.block_size, cache.heads, cache.head_dim, cache.fmt) == (4, 16, 2, 64, "mxfp4")
    assert cache.k_tscale is None and cache.v_tscale is None and cache.device == cache.k_codes.device
    assert (rope.rot_dim, rope.amplitude, rope.interleaved) == (32, 1.0, False)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_tensors_with_other_memory(nv, fmt):  # noqa: F811
    rng = np.random.default_rng(600)
    nb, table, lens, start = make_batch(rng, [40, 7], [1, 1], 16)
    one, two = (device_cache(nv, fmt, make_cache(rng, fmt, nb, 16, 2, 64)) for _ in range(2))
    q, k = rand(rng, (2, 4, 64), torch.float16), rand(rng, (2, 2, 64), torch.float16)
    freqs = torch.from_numpy(K.frequencies(None, 32, 1e4)).cuda()
    rope, other = nv.Rope(freqs.clone()), nv.Rope(freqs * 3)
    pos = i32([5, 90])

    def step(cache, rope):
        nv.kv_append(k, k, cache, i32(table), i32(lens), rope=rope)
        return nv.kv_attention(nv.rope(q, pos, rope), cache, i32(table), i32(lens))
    before, want = step(one, rope), step(two, other)
    assert not torch.equal(before, want)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales") + (("k_tscale", "v_tscale") if fmt == "nvfp4" else ()):
        getattr(one, name).data = getattr(two, name).clone()
    rope.freqs.data = other.freqs.clone()
    assert torch.equal(step(one, rope), want)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(two, name))
    one.v_codes.data = one.v_codes[:1].clone()
    with pytest.raises(ValueError):
        step(one, rope)
