"""Pins of the MXFP4 oracle: hand-worked blocks, closed forms and invariants."""
import numpy as np
import pytest

from oracle import mx


def _block(values):
    y = np.zeros((1, 128))
    y[0, :len(values)] = values
    return y


def test_hand_worked_block():
    # largest 7: floor(log2 7) = 2, E = 0; every border between codes, and its sign
    y = _block([7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.26, 0.74, 1.26, 5.01, 6.5, -0.1])
    codes, s = mx.quantize(y)
    assert s[0].tolist() == [127, 0, 0, 0]
    assert codes[0, :17].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 1, 3, 7, 7, 8]
    assert mx.values(codes, s)[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


@pytest.mark.parametrize("top,byte", [(4.0, 127), (3.999, 126), (8.0, 128), (7.999, 127), (1.0, 125), (2.0 ** -125, 0),
                                      (2.0 ** -126, 0), (2.0 ** -140, 0), (2.0 ** 127, 252), (2.0 ** 130, 254),
                                      (0.0, 0)])
def test_scales(top, byte):
    assert mx.quantize(_block([top]))[1][0, 0] == byte


def test_scales_of_small_blocks_leave_the_codes_smaller():
    # 2^-127 is the least scale: 2^-126 is 2 of it
    codes, s = mx.quantize(_block([2.0 ** -126, 2.0 ** -127, 2.0 ** -129]))
    assert codes[0, :3].tolist() == [4, 2, 0] and s[0, 0] == 0


def test_not_finite():
    y = _block([1.0, np.nan, 2.0])
    y[0, 40], y[0, 70] = np.inf, -np.inf
    codes, s = mx.quantize(y)
    assert s[0].tolist() == [255, 255, 255, 0] and not codes.any()
    assert np.isnan(mx.values(codes, s)[0, :96]).all()


def test_pack_bytes():
    codes = np.arange(16, dtype=np.uint8)[None]
    assert mx.pack(codes)[0].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert np.array_equal(mx.unpack(mx.pack(codes)), codes)


def test_scale_order():
    s = np.arange(24, dtype=np.uint8).reshape(3, 8)
    o = mx.scale_order(s)
    assert o.shape == (2, 3, 4)
    for r in range(3):
        for b in range(8):
            assert o[b // 4, r, b % 4] == s[r, b]


def test_properties():
    rng = np.random.default_rng(3)
    y = rng.standard_normal((40, 256)) * np.exp(3 * rng.standard_normal((40, 1)))
    codes, s = mx.quantize(y)
    v = mx.values(codes, s)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    a = np.abs(y) / scale
    assert (a < 8).all() and (a.reshape(40, -1, 32).max(-1) >= 4).all()
    # half a step: 1/4 below 2, 1/2 below 4, 1 up to 6, and up to 2 where it saturates
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    assert (np.abs(v - y) <= half * scale * (1 + 1e-12)).all()
    again, s2 = mx.quantize(v)
    assert np.array_equal(mx.values(again, s2), v)  # values of the format stay
    up, s3 = mx.quantize(8 * y)
    assert np.array_equal(up, codes) and np.array_equal(s3, s + 3)
    neg, s4 = mx.quantize(-y)
    assert np.array_equal(neg, codes ^ 8) and np.array_equal(s4, s)


def test_rotation_keeps_products():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((5, 512)), rng.standard_normal((7, 512))
    signs = rng.choice([-1, 1], 512)
    for block in (1, 128, 256, 512):
        y = mx.rotate(x, block, signs) @ mx.rotate(w, block, signs).T
        assert np.allclose(y, x @ w.T, atol=1e-10)
    one = np.zeros((1, 256))
    one[0, 3] = 16.0
    assert np.allclose(np.abs(mx.rotate(one, 256)), 1.0)


def test_gemm_by_hand():
    ca, cw = np.zeros((1, 128), np.uint8), np.zeros((2, 128), np.uint8)
    ca[0, 0], ca[0, 33] = 7, 11          # 6, -1.5
    cw[0, 0], cw[1, 33] = 9, 2           # -0.5, 1
    sa = np.array([[128, 126, 127, 127]], np.uint8)                        # 2, 1/2
    sw = np.array([[130, 0, 0, 0], [127, 129, 255, 127]], np.uint8)         # 8; 4 and a NaN block
    y, size = mx.gemm(ca, sa, cw, sw)
    assert y[0, 0] == 6 * 2 * -0.5 * 8 and size[0, 0] == 48 and np.isnan(y[0, 1])
