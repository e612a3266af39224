"""Limits of the MXFP4 calls that the header states, refused on the host (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

rw4 = pytest.importorskip("rotated_w4a4_amd", reason="librw4.so not built")

lib = rw4.lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, SHAPE = range(3)
P = 0x10000  # 16-byte aligned, never dereferenced


@pytest.mark.parametrize("block,N,K", [(1, 1 << 28, 512), (1, (1 << 14) - 1, 1 << 23), (128, 1 << 28, 512),
                                       (256, 1 << 28, 1024), (512, (1 << 25) - 5, 8192), (1, 16777153, 8192)])
@pytest.mark.parametrize("strides", ["kn", "apart"])
def test_weights_of_too_many_values(block, N, K, strides):
    # other layouts than [N, K] by 16-byte rows: one block for 64 x 128 values (64 x 256, 32 x 512), fewer than 2^24 blocks
    sk, sn = {"kn": (N, 1), "apart": (2, 2 * K)}[strides]
    t = ctypes.c_void_p()
    if block > 1:
        assert lib.rw4_transform_hadamard(K, block, None, ctypes.byref(t)) == OK
    try:
        assert lib.rw4_mx_pack_weight(t, P, 1, N, K, sk, sn, P, P, None) == SHAPE
    finally:
        if block > 1:
            lib.rw4_transform_destroy(t)


def test_grids(tmp_path):
    src = tmp_path / "check.cpp"
    src.write_text('#include "mx_index.h"\nusing namespace rw4;\n' + """
static_assert(mx_pack_blocks(64, 128, 1) == 1 && mx_pack_blocks(65, 256, 128) == 4 && mx_pack_blocks(64, 256, 256) == 1);
static_assert(mx_pack_blocks(33, 512, 512) == 2 && mx_pack_blocks(1, 384, 128) == 3);
// 2^37 values of 64 x 128 each are the first that do not fit; the largest operands leave no type
static_assert(mx_pack_blocks(1 << 14, 1 << 23, 1) == kMxPackMostBlocks + 1);
static_assert(mx_pack_blocks((1 << 14) - 64, 1 << 23, 1) <= kMxPackMostBlocks);
static_assert(mx_pack_blocks(1 << 28, 1 << 23, 1) > kMxPackMostBlocks);
static_assert(mx_gemm_fits(1 << 19, 1 << 19, 128) && !mx_gemm_fits((1 << 19) + 1, 1 << 19, 128));
static_assert(mx_gemm_fits(1, 1 << 28, 128) && mx_gemm_fits(1 << 28, 1, 128) && mx_gemm_fits(1 << 28, 1024, 128));
// from 1793 large tiles on they always fill 7/8 of their rounds: the 128 x 128 kernel has fewer than 2^13
constexpr bool filled() {
  for (int64_t tiles = 1793; tiles < 1 << 14; ++tiles)
    if (8 * tiles < 7 * 256 * ((tiles + 255) / 256)) return false;
  return true;
}
static_assert(filled());
static_assert(kMxPackMostBlocks * 256 < int64_t(1) << 32);
""")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-fsyntax-only", "-I", os.path.join(ROOT, "rotated_w4a4_amd", "csrc"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("M,N", [(1 << 28, 1 << 28), (1 << 20, (1 << 18) + 1), (1 << 28, 1025), (1025, 1 << 28)])
def test_products_of_too_many_values(M, N):
    # more than 2^22 tiles of 256 x 256, which is the kernel that they go to
    assert -(-M // 256) * -(-N // 256) > 1 << 22
    assert lib.rw4_mx_gemm(P, P, P, P, M, N, 128, P, 1, N, None) == SHAPE
