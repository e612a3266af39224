"""The choice of whole units for attention with sinks, compiled for the host (no GPU needed): evaluated in constant
expressions, where an overflow is an error."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _compile(tmp_path, body):
    src = tmp_path / "check.cpp"
    src.write_text('#include "kv_index.h"\nusing namespace rw4;\n' + body)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-fsyntax-only", "-I", os.path.join(ROOT, "rotated_w4a4_amd", "csrc"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_whole_units_of_few_rows(tmp_path):
    _compile(tmp_path, """
// 100 requests of 8 heads, each 17 steps, on 768 blocks: an equal share is 18 steps, whole units are 17
static_assert(whole_few(800, 256, 1000, 17, 800 * 17, 768));
// fewer units than wanted, more than the grid has blocks, or none wanted
static_assert(!whole_few(255, 256, 1000, 17, 255 * 17, 768) && !whole_few(1001, 256, 1000, 17, 1001 * 17, 768));
static_assert(!whole_few(800, 0, 1000, 17, 800 * 17, 768));
// one unit much longer than a share: 2 x share + 8 steps at most
static_assert(whole_few(800, 256, 1000, 44, 800 * 17, 768) && !whole_few(800, 256, 1000, 45, 800 * 17, 768));
// the longest requests that can be: nothing leaves its type
static_assert(whole_few(int64_t(1) << 23, 256, int64_t(1) << 23, 1 << 24, int64_t(1) << 47, 768));
static_assert(even_most((int64_t(1) << 47) / 768) > (int64_t(1) << 37));
static_assert(even_most(1) == 10);
""")


def test_lengths_of_a_tile_with_sinks_stay_in_32_bits(tmp_path):
    # positions of a tile: at most the request's keys, whatever sinks and window say
    _compile(tmp_path, """
constexpr int64_t most(int64_t sinks, int64_t window, int64_t tokens) {
  return ((sinks + 15) & ~int64_t(15)) + window + tokens + 15;
}
static_assert(((int64_t(kMostKeys) + 15) & ~int64_t(15)) <= 0x7FFFFFFF, "rounding the sinks up stays in an int");
static_assert(most(kMostKeys, int64_t(1) << 40, 1 << 25) > kMostKeys, "then the request's own length is the limit");
""")
