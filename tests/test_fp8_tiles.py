"""The E4M3 GEMM's index arithmetic and plans (csrc/fp8_tiles.hpp, which the kernel and its launches include) run on the
CPU under AddressSanitizer and UndefinedBehaviorSanitizer: tests/sanitize/fp8_tiles_driver.cpp checks every load, LDS
address, tile and zero row of the launches that real plans make.  A planted mistake in a copy of the header fails it."""
import os
import shutil
import subprocess

import pytest

from nvfp4_weight_only_amd import build as B

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize", "fp8_tiles_driver.cpp")
HEADER = os.path.join(B.CSRC, "fp8_tiles.hpp")


def run(tmp_path, planted=None):
    text = open(HEADER).read()
    if planted is not None:
        assert text.count(planted[0]) == 1, planted[0]
        text = text.replace(*planted)
    (tmp_path / "fp8_tiles.hpp").write_text(text)
    gxx, exe = shutil.which("g++"), str(tmp_path / "fp8_tiles_driver")
    if gxx is None:
        pytest.skip("g++ not found")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                    str(tmp_path), DRIVER, "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"),
                          timeout=300)


def test_fp8_gemm_indices_in_bounds(tmp_path):
    r = run(tmp_path)
    assert r.returncode == 0 and "checks" in r.stdout, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("planted", [
    ("return r < rows ? r : rows - 1;", "return r <= rows ? r : rows - 1;"),                  # a row past the last one
    ("(uint32_t)(16 * piece - (ktail - 16))", "(uint32_t)(16 * piece - ktail)"),              # the short chunk
    ("16 * piece >= ktail", "16 * piece > ktail"),
    ("return (uint32_t)(1024 * w + 8192 * j);", "return (uint32_t)(1024 * w + 4096 * j);"),   # LDS destinations
    ("return (lane & 7) ^ lane_row(lane);", "return lane & 7;"),                              # the swizzle
    ("16 * ((2 * g) ^ (l16 & 7))", "16 * ((2 * g) ^ (l16 & 3))"),
    ("(xcd < more ? xcd : more)", "(xcd < more ? more : xcd)"),                              # tiles of an XCD
    ("return used * xcd >> 3;", "return (used >> 3) * xcd;"),
    ("return xcd * m_tiles - t0 + mt - tn;", "return xcd * m_tiles - t0 + mt;"),              # zero rows
    ("(experts < pairs ? experts : pairs) + 7) / 8", "(experts < pairs ? experts : pairs)) / 8"),
    ("return Line{false, r < tm ? r : tm - 1};", "return Line{false, r};"),                   # lines ahead
    ("return c + kAhead < last ? c + kAhead : last;", "return c + kAhead;"),
    ("*in = o <= k - 16;", "*in = o <= k;"),                                                  # sums done again
    ("(int64_t)kb * slice / slices", "(int64_t)kb / slices * slice"),                         # chunks of a slice
], ids=range(14))
def test_fp8_gemm_planted_index_mistakes_are_found(tmp_path, planted):
    assert run(tmp_path, planted).returncode != 0
