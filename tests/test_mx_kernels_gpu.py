"""Every kernel of mx_gemm (mx_shapes.py) against the float64 oracle: scales of their own in each block, both output
types, rows of 16-byte multiples and others, what lies behind the rows and between them, ends of the scales."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import mx as omx  # noqa: E402
from tests.mx_shapes import ALL, SHAPES  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import DEV, dev, np64  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def _operand(rng, rows, K, low=123, high=132):
    return rng.integers(0, 16, (rows, K)).astype(np.uint8), rng.integers(low, high, (rows, K // 32)).astype(np.uint8)


def _stored(c, s):
    return dev(omx.pack(c)), dev(omx.scale_order(s))


def _product(a, w, dtype, pitch):
    """The product as [M, N] of a wider tensor, whose other values have to stay."""
    M, N = a[0].shape[0], w[0].shape[0]
    wide = torch.full((M + 1, pitch), 7.0, dtype=dtype, device=DEV)
    rw4.mx_gemm(*a, *w, out=wide[:M, :N])
    assert (wide[M:] == 7.0).all() and (wide[:, N:] == 7.0).all()
    return np64(wide[:M, :N])


def _pitches(N):
    """One of 16-byte multiples in both types, and an odd one."""
    return (N + 7) // 8 * 8 + 8, N + 3 - N % 2


@pytest.mark.parametrize("kernel,M,N,K", ALL)
def test_scales_of_every_block(kernel, M, N, K):
    rng = np.random.default_rng(M + 3 * N + K)
    (ca, sa), (cw, sw) = _operand(rng, M, K), _operand(rng, N, K)
    want, size = omx.gemm(ca, sa, cw, sw)
    a, w = _stored(ca, sa), _stored(cw, sw)
    # K exact products added in fp32, each addition off by at most one unit in the last place (2^-23) of a partial sum
    # that `size` bounds; then the output's own rounding
    sums = K * 2.0 ** -23 * size
    for dtype in (BF16, F32):
        for pitch in _pitches(N):
            err = np.abs(_product(a, w, dtype, pitch) - want)
            tol = sums + torch.finfo(dtype).eps / 2 * (np.abs(want) + sums)
            assert (err <= tol).all(), (dtype, pitch, int((err > tol).sum()), float((err - tol).max()))


@pytest.mark.parametrize("kernel,M,N,K", ALL)
def test_one_block_of_every_row(kernel, M, N, K):
    # a row's codes are zero outside one block, every block has a scale of its own: each output is one block's product or
    # zero, which fp32 holds exactly
    rng = np.random.default_rng(M + N + K)
    blocks = K // 32
    (ca, sa), (cw, sw) = _operand(rng, M, K, 100, 150), _operand(rng, N, K, 100, 150)
    for c, at in ((ca, rng.integers(0, blocks, len(ca))), (cw, np.arange(len(cw)) % blocks)):
        c.reshape(len(c), blocks, 32)[np.arange(blocks)[None] != at[:, None]] = 0
    want, _ = omx.gemm(ca, sa, cw, sw)
    a, w = _stored(ca, sa), _stored(cw, sw)
    for pitch in _pitches(N):
        assert np.array_equal(_product(a, w, F32, pitch), want), pitch
        rounded = np64(torch.from_numpy(want).to(BF16))
        assert np.array_equal(_product(a, w, BF16, pitch), rounded), pitch


@pytest.mark.parametrize("kernel", list(SHAPES))
def test_rows_and_columns_of_nan(kernel):
    # a scale of 255 in one block makes its row (column) NaN, all of it and nothing else
    M, N, K = max(SHAPES[kernel])
    rng = np.random.default_rng(12)
    (ca, sa), (cw, sw) = _operand(rng, M, K), _operand(rng, N, K)
    sa[M - 1, K // 32 - 1] = sw[N // 2, 0] = 255
    want, size = omx.gemm(ca, sa, cw, sw)
    for dtype, pitch in zip((BF16, F32), _pitches(N)):
        got = _product(_stored(ca, sa), _stored(cw, sw), dtype, pitch)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        keep = ~np.isnan(want)
        sums = K * 2.0 ** -23 * size[keep]
        assert (np.abs(got[keep] - want[keep]) <= sums + torch.finfo(dtype).eps / 2 * (np.abs(want[keep]) + sums)).all()


@pytest.mark.parametrize("kernel", list(SHAPES))
def test_scales_far_apart(kernel):
    # exponents at both ends whose sums are ordinary: 2^127 times 2^-126 .. 2^-108 along some rows, the reverse along others
    M, N, K = max(SHAPES[kernel])
    rng = np.random.default_rng(13)
    ca, cw = _operand(rng, M, K)[0], _operand(rng, N, K)[0]
    sa, sw = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    sa[:, 0], sw[:, 0] = 254, rng.integers(1, 20, N)
    sa[:, -1], sw[:, -1] = rng.integers(1, 20, M), 254
    if K // 32 > 4:
        sa[:, 3], sw[:, 3] = 254, 0
    want, size = omx.gemm(ca, sa, cw, sw)
    got = _product(_stored(ca, sa), _stored(cw, sw), F32, _pitches(N)[0])
    sums = K * 2.0 ** -23 * size
    assert (np.abs(got - want) <= sums + 2.0 ** -24 * (np.abs(want) + sums)).all()
