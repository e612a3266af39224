"""The INT4 KV cache's serving operators at the ends of their ranges."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import oracle  # noqa: E402
from oracle import kv as okv  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests import kv_util as ku  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("hint", [1, 70])
def test_attention_longest_lengths(hint):
    # lengths up to the largest 32-bit number, on a table that has room for them, are clamped to 2^31 - 8192 keys; the
    # window shows the last of them, which are those of a short request that ends in the same page
    rng = np.random.default_rng(31)
    D, page, pages, hk, window = 64, 1 << 20, 2, 1, 5000
    cache = rw4.KVCache.empty(pages, page, hk, D)
    last = page - 8192  # keys of the last page
    T = window + hint
    k, v = (ku.dev(rng.standard_normal((T, hk, D)).astype(np.float32), BF16) for _ in range(2))
    rw4.kv_append(cache, k, v, ku.dev((page + last - T + np.arange(T)).astype(np.int64)))
    q = ku.dev(rng.standard_normal((hint, 2, D)).astype(np.float32), BF16)
    cu = ku.dev(np.array([0, hint], np.int32))
    want = rw4.kv_attention(q, cache, ku.dev(np.array([[1]], np.int32)), ku.dev(np.array([last], np.int32)), cu,
                            max_q_len=hint, window=window)
    table = np.zeros((1, 2048), np.int32)
    table[0, -1] = 1
    for length in (2 ** 31 - 8192, 2 ** 31 - 4000, 2 ** 31 - 1):
        got = rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array([length], np.int32)), cu, max_q_len=hint,
                               window=window)
        assert torch.equal(got, want) and torch.isfinite(got).all() and (got != 0).any(), length


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32), (128, F32), (256, F32)])
@pytest.mark.parametrize("rows", [2, 140])
def test_attention_scales_that_are_not_finite(D, dtype, rows):
    # one key with a scale that is not finite, of the key or of the value alone, under products of both signs: rows that
    # see it are NaN, the others as without it
    rng = np.random.default_rng(32)
    page, n, bad = 16, 200 + rows, 150 + rows
    pages = -(-n // page)
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    table, kv = ku.dev(np.arange(pages, dtype=np.int32)[None]), ku.dev(np.array([n], np.int32))
    cu = ku.dev(np.array([0, rows], np.int32))
    q = rng.standard_normal((rows, 2, D)).astype(np.float32)
    q[:, 0] = 0.3 * ck[bad // page, 0, bad % page]  # a product above zero
    q[:, 1] = -q[:, 0]
    q = ku.dev(q, dtype)
    window = 60  # the last rows see the key, the rows behind it and those in front of it do not
    cases = [(x, None) for x in (np.inf, -np.inf, np.nan)] + [(None, x) for x in (np.inf, -np.inf, np.nan)]
    place = n - rows + np.arange(rows)
    see = torch.from_numpy((place >= bad) & (place - window < bad))
    assert see.any()
    x, lse = rw4.kv_attention(q, ku.cache_of(ck, sk, cv, sv), table, kv, cu, max_q_len=rows, window=window,
                              return_lse=True)
    assert torch.isfinite(x).all()
    for k_scale, v_scale in cases:
        sk2, sv2 = sk.copy(), sv.copy()
        if k_scale is not None:
            sk2[bad // page, 0, bad % page] = k_scale
        if v_scale is not None:
            sv2[bad // page, 0, bad % page] = v_scale
        y, lse2 = rw4.kv_attention(q, ku.cache_of(ck, sk2, cv, sv2), table, kv, cu, max_q_len=rows, window=window,
                                   return_lse=True)
        y, lse2 = y.cpu(), lse2.cpu()
        assert torch.isnan(y[see]).all(), (k_scale, v_scale)
        assert torch.equal(y[~see], x.cpu()[~see]) and torch.equal(lse2[~see], lse.cpu()[~see]), (k_scale, v_scale)
