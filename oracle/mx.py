"""CPU oracle of the MXFP4 calls (numpy float64) -- test infrastructure, written
from the definitions: dense Hadamard products, distances to the eight values, no
shared code with the HIP path."""
from __future__ import annotations

import numpy as np

from .reference import hadamard

__all__ = ["VALUES", "rotate", "quantize", "pack", "unpack", "scale_order", "values", "gemm",
           "quantize_whole"]

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rotate(x, block, signs=None):
    """x R in float64 (block 1: x)."""
    x = np.asarray(x, np.float64)
    if block == 1:
        return x
    if signs is not None:
        x = x * np.asarray(signs, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = x.reshape(-1, block) @ hadamard(block)
        return (y / np.sqrt(float(block))).reshape(x.shape)


def quantize(y):
    """Codes (0..15) [rows, K] and scale bytes [rows, K / 32] of y [rows, K]."""
    rows, K = y.shape
    b = y.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -127)
    e[top > 0] = np.clip(np.floor(np.log2(top[top > 0])).astype(int), -200, 200)
    # log2 rounds: the power of two is checked against the number itself
    e[top > 0] += (np.ldexp(1.0, e[top > 0] + 1) <= top[top > 0]).astype(int)
    e[top > 0] -= (np.ldexp(1.0, e[top > 0]) > top[top > 0]).astype(int)
    e = np.where(top > 0, np.clip(e - 2, -127, 127), -127)
    a = np.ldexp(np.abs(b), -e[..., None])
    # nearest of the values; of two at the same distance the one with the even index
    dist = np.abs(a[..., None] - VALUES)
    near = dist == dist.min(-1, keepdims=True)
    index = np.where((near & (np.arange(8) % 2 == 0)).any(-1), (near & (np.arange(8) % 2 == 0)).argmax(-1), near.argmax(-1))
    codes = (index | ((b < 0) << 3)).astype(np.uint8).reshape(rows, K)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def pack(codes):
    """Bytes [rows, K / 2], the even channel in the low four bits."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def scale_order(s):
    """Scale bytes [rows, K / 32] in the stored order [K / 128, rows, 4]."""
    rows, blocks = s.shape
    return np.ascontiguousarray(s.reshape(rows, blocks // 4, 4).transpose(1, 0, 2))


def values(codes, s):
    """float64 values [rows, K] of codes and scale bytes by rows (255: NaN)."""
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(int) - 127))
    rows, K = codes.shape
    return (v.reshape(rows, -1, 32) * scale[..., None]).reshape(rows, K)


def gemm(ca, sa, cw, sw):
    """(Y, the sums of the products' sizes), float64."""
    a, w = values(ca, sa), values(cw, sw)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def quantize_whole(x, block, unit):
    """Codes and scale bytes of x R for x of whole numbers (int64 [rows, K], sums below 2^63) times 2^unit, in whole
    numbers throughout: |y| against a border t is u^2 against t^2 block."""
    rows, K = x.shape
    u = (x.reshape(rows, -1, block) @ hadamard(block).astype(np.int64)).reshape(rows, K)
    codes, scales = np.zeros((rows, K), np.uint8), np.zeros((rows, K // 32), np.uint8)

    def at_least(n, quarters, e):
        """(-1, 0, 1) as n / sqrt(block) is below, at or above quarters 2^(e - 2), n >= 0."""
        left, right, e = n * n, quarters * quarters * block, 2 * (e - 2)
        left, right = (left, right << e) if e >= 0 else (left << -e, right)
        return (left > right) - (left < right)

    for r in range(rows):
        for b in range(K // 32):
            part = [int(v) for v in u[r, 32 * b:32 * b + 32]]
            top = max(abs(v) for v in part)
            e = -127 - unit
            if top > 0:
                two = top.bit_length()  # 2^two > top >= top / sqrt(block)
                while at_least(top, 4, two) < 0:
                    two -= 1
                e = max(-127, min(127, two - 2 + unit)) - unit
            scales[r, b] = e + unit + 127
            for i, v in enumerate(part):
                code = 0
                for k, quarters in enumerate((1, 3, 5, 7, 10, 14, 20)):  # between code k and k + 1; a tie to the even one
                    side = at_least(abs(v), quarters, e)
                    code += side > 0 or (side == 0 and k % 2 == 1)
                codes[r, 32 * b + i] = code | (8 if v < 0 else 0)
    return codes, scales
