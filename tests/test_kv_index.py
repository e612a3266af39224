"""Index arithmetic of the KV cache kernels, compiled for the host (no GPU
needed): evaluated in constant expressions, where an overflow is an error."""
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


def test_page_ids_of_the_longest_requests_stay_in_the_table(tmp_path):
    # every length a table can hold and more: a lane reads entry j / page_size only for j in [0, keys), for the first
    # tile of every group that starts in front of the last key
    _compile(tmp_path, """
constexpr bool lanes_fit(int64_t len, int64_t room) {
  const int hi = clamp_keys(len, room);
  if (hi < 0 || hi > room) return false;
  for (int back = 1; back <= 4500; back += back < 200 ? 1 : 61) {
    const int j = hi - back;
    if (j < 0) break;
    for (int lane = 0; lane < 64; ++lane) {
      const int key = j + ids_ahead(lane);
      if (key < j) return false;
    }
    const int next = j + 128 + 64 + 127;  // two steps ahead of the kernel for many rows, rows of a step behind
    if (next < j) return false;
  }
  return true;
}
static_assert(lanes_fit(0x7FFFFFFF, int64_t(2048) << 20));
static_assert(lanes_fit(0x7FFFFFFF, int64_t(0x7FFFFFFF) << 20));
static_assert(lanes_fit(0x7FFFFF00, int64_t(2048) << 20));
static_assert(lanes_fit(-5, 64) && lanes_fit(100, 64) && lanes_fit(1 << 20, 0));
static_assert(clamp_keys(-1, 64) == 0 && clamp_keys(100, 64) == 64 && clamp_keys(63, 64) == 63);
""")


def test_whole_units_only_where_none_outlasts_a_share(tmp_path):
    _compile(tmp_path, """
// 4 prompts of 1500..2048 tokens (8 heads, group 4): 1800 units of 24..32 steps on 512 blocks
static_assert(whole_units(1800, 1024, 1800, 32, 1800 * 28, 512));
static_assert(whole_units(1024, 1024, 2000, 32, 1024 * 32, 512));
static_assert(!whole_units(1023, 1024, 2000, 32, 1023 * 32, 512) && !whole_units(1 << 20, 0, 1 << 20, 1, 1 << 20, 512));
// one chunk of 256 tokens on 65536 keys (64 units of 1024 steps) beside 63 prompts of 128 (2016 units of 2): a share
// is 136 steps, whole units would take 1024
static_assert(!whole_units(64 + 2016, 1024, 3000, 1024, 64 * 1024 + 2016 * 2, 512));
static_assert(whole_units(int64_t(1) << 23, 1024, int64_t(1) << 23, 1 << 24, int64_t(1) << 47, 768));
// no block for every unit: equal shares; and no grid of 2^32 threads
static_assert(!whole_units(1801, 1024, 1800, 32, 1801 * 28, 512));
static_assert(wide_grid(1800, 512) == 1800 && wide_grid(100, 512) == 512 && wide_grid(int64_t(1) << 24, 768) == 768);
static_assert(256 * wide_grid((int64_t(1) << 24) - 1, 768) < int64_t(1) << 32);
""")


def test_workspace_goes_by_the_kernels_a_call_can_get():
    rw4 = pytest.importorskip("rotated_w4a4_amd", reason="librw4.so not built")
    ws = rw4.lib.rw4_kv_attention_workspace_bytes
    for D, few, few_mb, mb in ((64, 32, 7, 52), (128, 48, 13, 69), (256, 48, 17, 68)):
        rows = few // 4
        assert ws(1, 1, 32, 8, D) == ws(rows, rows, 32, 8, D) <= few_mb * 10 ** 6
        assert ws(1, 1, 32, 8, D) < ws(rows + 1, 1, 32, 8, D) == ws(10 ** 6, 9, 32, 8, D) <= mb * 10 ** 6
