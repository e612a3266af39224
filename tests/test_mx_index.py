"""The choice of the MXFP4 product's kernel, compiled for the host (no GPU needed): evaluated in constant expressions,
where an overflow is an error."""
import os
import shutil
import subprocess

import pytest

from tests.mx_shapes import ALL, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _compile(tmp_path, body):
    src = tmp_path / "check.cpp"
    src.write_text('#include "mx_index.h"\nusing namespace rw4;\n' + body)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-fsyntax-only", "-I", os.path.join(ROOT, "rotated_w4a4_amd", "csrc"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_every_kernel_has_shapes(tmp_path):
    # a kernel without a shape leaves the switch incomplete
    _compile(tmp_path, "#pragma GCC diagnostic error \"-Wswitch\"\nint f(MxKernel k) {\n  switch (k) {\n"
             + "".join(f"    case MxKernel::{k}: return {len(v)};\n" for k, v in SHAPES.items() if v) + "  }\n  return 0;\n}\n")


def test_shapes_take_their_kernel(tmp_path):
    _compile(tmp_path, "".join(f"static_assert(mx_kernel_for({M}, {N}, {K}) == MxKernel::{kernel});\n"
                               for kernel, M, N, K in ALL))


def test_largest_operands(tmp_path):
    _compile(tmp_path, """
constexpr int64_t rows = int64_t(1) << 28, longest = int64_t(1) << 23;
static_assert(mx_kernel_for(rows, rows, longest) == MxKernel::Tile256);
static_assert(mx_kernel_for(1, rows, 128) == MxKernel::Tile256 && mx_kernel_for(1, int64_t(1) << 26, 128) == MxKernel::Few2);
// single tokens: the grid they are given holds every channel
static_assert(((int64_t(1) << 26) + kMxFewChannels - 1) / kMxFewChannels <= kMxMostBlocks);
""")


def test_shapes_of_the_longest_rows_take_their_kernel(tmp_path):
    from tests.test_mx_longest_gpu import K, SHAPES as longest
    _compile(tmp_path, "".join(f"static_assert(mx_kernel_for({M}, {N}, {K}) == MxKernel::{k});\n"
                               for k, (M, N) in longest.items()))
