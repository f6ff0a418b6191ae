"""Which tokens a row of attention sees (csrc/kv_masks.hpp, which the kernels include) on the CPU under AddressSanitizer
and UndefinedBehaviorSanitizer, up to windows and positions of 2^31 - 1 (tests/sanitize/kv_masks_driver.cpp).  A planted
mistake in a copy of the header fails it, among them differences that pass 32 bits."""
import os
import shutil
import subprocess

import pytest

from nvfp4_weight_only_amd import build as B

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize", "kv_masks_driver.cpp")


def run(tmp_path, planted=None):
    text = open(os.path.join(B.CSRC, "kv_masks.hpp")).read()
    if planted is not None:
        assert text.count(planted[0]) == 1, planted[0]
        text = text.replace(*planted)
    (tmp_path / "kv_masks.hpp").write_text(text)
    gxx, exe = shutil.which("g++"), str(tmp_path / "kv_masks_driver")
    if gxx is None:
        pytest.skip("g++ not found")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                    str(tmp_path), DRIVER, "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"),
                          timeout=300)


def test_seen_tokens(tmp_path):
    r = run(tmp_path)
    assert r.returncode == 0 and "checks" in r.stdout, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("planted", [
    ("(window > 0 && to > window ? low_bits(to - window) : 0u)", "(window > 0 ? low_bits(pos - window - t0 + 1) : 0u)"),
    ("low_bits(to - window)", "low_bits(to - window + 1)"),
    ("return t <= pos &&", "return t < pos &&"),
    ("const int32_t to = pos - t0 + 1;", "const int32_t to = pos - t0;"),
    ("pos - t < window", "pos - t <= window"),
    ("pos >= window ? pos - window + 1 : 0", "pos > window ? pos - window + 1 : 0"),
    ("first < end ? first : end", "first"),
    ("const int64_t first = pos - window + 1;", "const int64_t first = pos - window + 32;"),
], ids=range(8))
def test_planted_mistakes_are_found(tmp_path, planted):
    assert run(tmp_path, planted).returncode != 0
