"""Inputs and comparisons of the KV cache tests."""
import numpy as np
import torch

import oracle
import rotated_w4a4_amd as rw4
from oracle import kv as okv

DEV = "cuda:0"
U24 = 2.0 ** -24


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if dtype is None else t.to(dtype)


def np64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def page_table(rng, lengths, page, width, pages):
    """A block table with the pages of each length, in random order; other cells hold a page out of range."""
    table = np.full((len(lengths), width), pages + 7, np.int32)
    ids = rng.permutation(pages)
    at = 0
    for b, n in enumerate(lengths):
        need = min(-(-n // page), width)
        table[b, :need] = ids[at:at + need]
        at += need
    return table


def pool(rng, pages, heads, page, D, spread=0.3):
    """Codes int8 [pages, heads, page, D] and scales fp32 of a cache half."""
    g = rng.standard_normal((pages, heads, page, D))
    m = np.abs(g).max(-1, keepdims=True)
    codes = np.rint(7 * g / m).astype(np.int8)
    scales = (m[..., 0] / 7 * np.exp(spread * rng.standard_normal((pages, heads, page)))).astype(np.float32)
    return codes, scales


def stored(codes):
    """The packed bytes of codes [..., D]."""
    return oracle.pack_int4(codes.reshape(-1, codes.shape[-1])).reshape(*codes.shape[:-1], codes.shape[-1] // 2)


def opened(packed):
    """Codes of a uint8 device tensor [..., D / 2] of any strides."""
    torch.cuda.synchronize()
    x = packed.cpu().contiguous().numpy()
    return oracle.unpack_int4(x.reshape(-1, x.shape[-1])).reshape(*x.shape[:-1], 2 * x.shape[-1])


def cache_of(ck, sk, cv, sv, layout="hnd"):
    """A KVCache of these codes and scales; layout "nhd": slots outside, heads inside."""
    parts = [dev(stored(ck)), dev(stored(cv)), dev(sk), dev(sv)]
    if layout == "nhd":
        parts = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in parts]
    return rw4.KVCache(*parts)


def close(got, want, tol, what):
    """Every |got - want| <= tol, with the same infinities."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), f"{what}: non-finite values differ"
    assert np.isfinite(got[fin]).all(), f"{what}: non-finite where the definition is finite"
    err = np.abs(got[fin] - want[fin])
    lim = np.broadcast_to(tol, want.shape)[fin]
    if err.size and not (err <= lim).all():
        i = int(np.argmax(err - lim))
        raise AssertionError(f"{what}: off by {err[i]:.3e}, allowed {lim[i]:.3e}, at {int((err > lim).sum())} places")


def attention_tolerance(out, reach, size, dtype, D, keys):
    """Allowed |error| of attention's output, from its roundings.

    Scores: a D-term fp32 sum and its scalings, (D + 4) 2^-24 of size; the softmax works on s - m, |s - m| <= 2 size,
    whose base-2 argument is rounded twice (2^-24 of it each), as an exponent an error of the same relative size;
    numerator and denominator: twice.  exp, the scale product, 2^-24 each, sums over `keys` keys (running rescales
    included) 2^-24 per addition along a chain no longer than the keys; bf16 output: probabilities rounded once to
    bf16.  All of it acts on reach; the fp32 tail (normalization, Hadamard, 1 / sqrt(D)) adds 12 2^-24 of reach, the
    output's own rounding acts on the value."""
    rel = 2 * ((D + 4) * U24 + 4 * U24) * size + (min(keys, 4096) + 24) * U24
    if dtype is torch.bfloat16:
        rel = rel + half_step(dtype)
    return rel[..., None] * reach[..., None] + half_step(dtype) * np.abs(out) + 1e-30
