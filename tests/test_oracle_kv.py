"""Pins of the KV cache oracle: closed forms and invariants (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import kv as okv


def test_slots_by_hand():
    # page 4; request 0 grows 3 -> 5 (one page), 1 fills its page 6 -> 8 (none), 2 finished (2 pages back),
    # 3 needs 2 pages and finds 1, 4 needs none and is served, 5 needs one after the list ran short
    table = np.full((6, 3), -1)
    table[0, 0], table[1, :2], table[2, :2], table[4, 0], table[3, 0] = 10, (11, 12), (13, 14), 15, 16
    ring = np.array([0, 20, 21, 0, 0, 0, 0])
    got = okv.kv_slots([3, 6, 8, 4, 1, 0], [2, 2, -1, 8, 1, 1], table, ring, [1, 2], 4, 16)
    kv_len, cu, served, slots, pos, table, ring, state = got
    assert kv_len.tolist() == [5, 8, 0, 4, 2, 0]
    assert cu.tolist() == [0, 2, 4, 4, 12, 13, 14]
    assert served.tolist() == [1, 1, 1, 0, 1, 0]
    assert slots[:4].tolist() == [43, 80, 50, 51] and (slots[4:12] == -1).all()
    assert slots[12] == 61 and slots[13] == -1 and (slots[14:] == -1).all()
    assert pos[:4].tolist() == [3, 4, 6, 7] and pos[12] == 1
    assert table[0, 1] == 20
    assert state.tolist() == [2, 3] and ring[3:5].tolist() == [13, 14]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_keeps_lengths_and_differences(interleaved):
    rng = np.random.default_rng(0)
    D, rot = 64, 32
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(50)[:, None] * f
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x, y = rng.standard_normal((2, 1, 1, D))

    def at(v, p):
        return okv.norm_rope(v, None, 0.0, table, np.array([p]), interleaved)[0][0, 0]

    assert np.isclose(np.linalg.norm(at(x, 17)), np.linalg.norm(x))
    assert np.array_equal(at(x, 17)[rot:], x[0, 0, rot:])
    assert np.isclose(at(x, 9) @ at(y, 4), at(x, 29) @ at(y, 24))  # depends on the distance alone
    assert np.allclose(at(x, 0), x[0, 0])


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(1).standard_normal((3, 2, 128)) * 5
    y, f = okv.norm_rope(x, np.ones(128), 0.0, None, None, False)
    assert np.allclose(((y * f) ** 2).mean(-1), 1.0)


def test_quantized_heads_are_the_oracles_groups():
    x = np.random.default_rng(2).standard_normal((5, 3, 128))
    codes, scales = okv.quantize_heads(x, np.ones((5, 3, 1)), True)
    want, sw, _ = oracle.quantize_groups(okv.rotate_heads(x).reshape(15, 128))
    assert np.array_equal(codes.reshape(15, 128), want) and np.allclose(scales.reshape(15, 1), sw)


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    D, P, pages = 64, 16, 4
    cv = rng.integers(-7, 8, (pages, 1, P, D)).astype(np.int8)
    sv = np.ones((pages, 1, P))
    table = np.array([[2, 0, 3]])
    # equal scores: the mean of the values in sight, lse = log n
    ck = np.zeros((pages, 1, P, D), np.int8)
    out, lse, _, _ = okv.kv_attention(np.ones((2, 1, D)), ck, sv, cv, sv, pages, table, [37], [0, 2], 1.0, True, 0,
                                      False)
    seq = np.concatenate([cv[2, 0], cv[0, 0], cv[3, 0]])
    assert np.allclose(out[0, 0], seq[:36].mean(0)) and np.allclose(out[1, 0], seq[:37].mean(0))
    assert np.allclose(lse[:, 0], np.log([36, 37]))
    # a window of one key gives that key's value; rotated, its rotation
    out, _, _, _ = okv.kv_attention(np.ones((1, 1, D)), ck, sv, cv, sv, pages, table, [37], [0, 1], 1.0, True, 1, True)
    assert np.allclose(out[0, 0], okv.rotate_heads(seq[36].astype(float)))
    # more queries than keys: rows before the first key are empty
    out, lse, _, _ = okv.kv_attention(np.ones((3, 1, D)), ck, sv, cv, sv, pages, table, [1], [0, 3], 1.0, True, 0,
                                      False)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], seq[0])
