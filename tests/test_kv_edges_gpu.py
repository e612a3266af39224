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
