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


def _weights_case(D, sv_of, score_of=None, n=300, q_len=90, unrotate=False, seed=33):
    """Attention of q_len rows on n keys with the value scales sv_of(rng, n) (and scores steered by score_of), in the
    kernel for many rows, against the oracle.  Allowed: 2^-11 of each weight (fp16; two bf16 parts are finer), the fp32
    terms of ku.attention_tolerance and the output's rounding.  What fp16 loses of small weights, 2^-25 a key, is less
    than 2^-14 of the largest weight in the cases that stay in it (n <= 20000, largest 2^4 or more)."""
    rng = np.random.default_rng(seed)
    page = 16
    pages = -(-n // page)
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    sv = sv_of(rng, pages * page).astype(np.float32).reshape(pages, 1, page)
    if score_of is not None:
        ck[:] = np.where(rng.random(ck.shape) < 0.5, -1, 1)
        ck[..., 0] = 7
        sk[:] = score_of(pages * page).astype(np.float32).reshape(pages, 1, page) / 7
    q = rng.standard_normal((q_len, 2, D))
    if score_of is not None:
        q[:] = 0
        q[..., 0] = 1  # the score of a key is its score_of
    q = ku.dev(q.astype(np.float32), BF16)
    table, cu = np.arange(pages, dtype=np.int32)[None], [0, q_len]
    scale = 1.0 if score_of is not None else D ** -0.5
    out, lse = rw4.kv_attention(q, ku.cache_of(ck, sk, cv, sv), ku.dev(table), ku.dev(np.array([n], np.int32)),
                                ku.dev(np.array(cu, np.int32)), max_q_len=q_len, unrotate=unrotate, scale=scale,
                                return_lse=True)
    want, wl, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, [n], cu, scale, True, 0, unrotate)
    rel = 2.0 ** -11 + 2 * (D + 8) * ku.U24 * size + (n + 24) * ku.U24
    tol = rel[..., None] * reach[..., None] + ku.half_step(BF16) * np.abs(want)
    ku.close(ku.np64(out), want, tol, "out")
    ku.close(ku.np64(lse), wl, (D + 8) * ku.U24 * size + (64 + n) * ku.U24 + 4 * ku.U24 * np.abs(wl), "lse")


@pytest.mark.parametrize("unrotate", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_rows_keep_their_weights(D, unrotate):
    _weights_case(D, lambda rng, n: np.exp(0.3 * rng.standard_normal(n)), unrotate=unrotate)


def _at(x, where, value):
    x[where] = value
    return x


VALUE_SCALES = {
    "tiny": lambda rng, n: 1e-30 * np.exp(0.3 * rng.standard_normal(n)),
    "huge": lambda rng, n: 1e30 * np.exp(0.3 * rng.standard_normal(n)),
    "far_apart": lambda rng, n: np.exp(6 * rng.standard_normal(n)),
    "further_apart": lambda rng, n: np.exp(np.clip(20 * rng.standard_normal(n), -50, 50)),
    "zeros": lambda rng, n: np.zeros(n),
    "some_zeros": lambda rng, n: np.exp(0.3 * rng.standard_normal(n)) * (rng.random(n) < 0.7),
    "first_step_zero": lambda rng, n: _at(np.exp(0.3 * rng.standard_normal(n)), slice(0, 64), 0.0),
    "first_small": lambda rng, n: _at(np.exp(0.3 * rng.standard_normal(n)), 0, 1e-9),
    "late_large": lambda rng, n: _at(np.exp(0.3 * rng.standard_normal(n)), n - 90, 3e7),
    "late_small": lambda rng, n: _at(np.exp(0.3 * rng.standard_normal(n)), n - 60, 1e-12),
    "rising": lambda rng, n: 2.0 ** (np.arange(n) / 8.0),
    "falling": lambda rng, n: 2.0 ** (-np.arange(n) / 8.0),
    "negative": lambda rng, n: np.exp(0.3 * rng.standard_normal(n)) * rng.choice([-1, 1], n),
}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", VALUE_SCALES)
def test_attention_many_rows_value_scales_of_any_range(name, D):
    _weights_case(D, VALUE_SCALES[name])


@pytest.mark.parametrize("D,n", [(64, 2000), (128, 2000), (128, 20000)])
@pytest.mark.parametrize("low", [-8.0, -14.0, -20.0])
@pytest.mark.parametrize("sink", [1.0, 1e-3, 0.0])
def test_attention_many_rows_tails_of_small_weights(D, n, low, sink):
    # one key takes the maximum, the others share what is left of the softmax, e^low each; the first key's value may be
    # small or zero, so that the tail makes the output
    _weights_case(D, lambda rng, k: _at(np.exp(0.1 * rng.standard_normal(k)), 0, sink),
                  lambda k: _at(low + 0.1 * np.sin(np.arange(k)), 0, 0.0), n=n, q_len=66)


def test_cache_of_one_head_or_page_with_other_strides():
    # the stride of a dimension of one entry says nothing: tensors that differ in it alone are a cache
    D, page, pages = 64, 16, 3
    k, v = (torch.zeros((pages, 1, page, D // 2), dtype=torch.uint8, device=ku.DEV) for _ in range(2))
    ks, vs = torch.zeros((pages, 1, page), device=ku.DEV), torch.zeros((pages, page), device=ku.DEV).unsqueeze(1)
    v2 = v.squeeze(1).as_strided((pages, 1, page, D // 2), (page * D // 2, 5, D // 2, 1))
    vs2 = vs.as_strided((pages, 1, page), (page, 77, 1))
    x = ku.dev(np.random.default_rng(0).standard_normal((pages * page, 1, D)).astype(np.float32))
    slots = torch.arange(pages * page, device=ku.DEV)
    for a, b in ((v, vs), (v2, vs2)):
        cache = rw4.KVCache(k, a, ks, b)
        rw4.kv_append(cache, x, x, slots)
        assert torch.equal(cache.k, cache.v) and torch.equal(cache.k_scale, cache.v_scale) and (ks > 0).all()
        a.zero_()
    with pytest.raises(ValueError, match="strides"):
        rw4.KVCache(k, v, ks, torch.zeros((page, pages), device=ku.DEV).t().unsqueeze(1))


# magnitudes of rows, and eps: squares that leave fp32's range at either end
MAGNITUDES = [(1e19, 1e-6), (3e25, 1e-6), (2e36, 1e-6), (1e-17, 0.0), (1e-25, 0.0), (1e-36, 0.0), (1e-25, 1e-30),
              (1e-20, 1e-38), (1e-30, 1e-6), (1e18, 1e30)]


def _rows_of(seed, T, heads, D, dtype, big):
    """Rows of magnitude `big`, every third of 1 and one of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, heads, D)) * np.where(np.arange(T) % 3 == 1, 1.0, big)[:, None, None]
    x[4] = 0
    return ku.dev(x.astype(np.float32), dtype)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("D,dtype,inter", [(64, BF16, False), (128, F32, False), (128, BF16, True), (256, F32, True)])
@pytest.mark.parametrize("big,eps", MAGNITUDES)
def test_norm_of_any_magnitude(big, eps, D, dtype, inter, rotate):
    # queries and keys through qk_norm_rope (also in place) and kv_append, against the oracle
    T, hq, hk, page = 11, 6, 3, 16
    rng = np.random.default_rng(34)
    q, k = _rows_of(1, T, hq, D, dtype, big), _rows_of(2, T, hk, D, dtype, big)
    v = _rows_of(3, T, hk, D, dtype, 1.0)
    w = (1 + 0.3 * rng.standard_normal((2, D))).astype(np.float32)
    wd = [ku.dev(x) for x in w]
    cs, pos = rw4.rope_table(50, D // 2), rng.integers(0, 50, T).astype(np.int32)
    kw = dict(eps=eps, interleaved=inter, rotate=rotate)
    got = rw4.qk_norm_rope(q, k, wd[0], wd[1], cs, ku.dev(pos), **kw)
    rows = [t for t in range(T) if eps > 0 or t != 4]  # 0 / 0 otherwise
    exact = []
    for x, y, wt in ((q, got[0], w[0]), (k, got[1], w[1])):
        z, f = okv.norm_rope(ku.np64(x)[rows], wt, float(np.float32(eps)), ku.np64(cs), pos[rows], inter)
        exact.append((z, f))
        want = okv.rotate_heads(z * f) if rotate else z * f
        # as for rows of ordinary size (32 roundings of the row's length and the output's own); below fp32's normal range
        # the roundings are of 2^-149
        tol = 32 * ku.U24 * np.linalg.norm(z * f, axis=-1, keepdims=True) + ku.half_step(dtype) * np.abs(want) + 2.0 ** -140
        ku.close(ku.np64(y)[rows], want, tol, "rows")
    q2, k2 = q.clone(), k.clone()
    rw4.qk_norm_rope(q2, k2, wd[0], wd[1], cs, ku.dev(pos), q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2[rows], got[0][rows]) and torch.equal(k2[rows], got[1][rows])
    cache = rw4.KVCache.empty(1, page, hk, D)
    q3 = rw4.kv_append(cache, k, v, torch.arange(T, device=ku.DEV), q, wd[0], wd[1], cs, ku.dev(pos), **kw)
    assert torch.equal(q3[rows], got[0][rows])
    z, f = exact[1]
    c, s = okv.quantize_heads(z, f, rotate)
    assert np.array_equal(ku.opened(cache.k)[0].transpose(1, 0, 2)[rows], c)
    ku.close(ku.np64(cache.k_scale)[0].T[rows], s, np.abs(s) * 18 * ku.U24 + 2.0 ** -140, "scale")
    assert (cache.k_scale[0, :, 4] == 0).all() and (ku.opened(cache.k)[0, :, 4] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotated_rows_at_the_end_of_the_range(D):
    # sums under the Hadamard pass fp32's range where the result does not; infinities and NaN stay in their rows
    T = 6
    rng = np.random.default_rng(35)
    x = rng.uniform(0.2, 0.5, (T, 3, D)) * 3e38
    x[0] = rng.standard_normal((3, D))
    q = ku.dev(x.astype(np.float32))
    got = rw4.qk_norm_rope(q, rotate=True)[0]
    want = okv.rotate_heads(ku.np64(q))
    fits = np.abs(want) < 3.4e38
    ku.close(ku.np64(got)[fits], want[fits], (32 * ku.U24 * np.linalg.norm(ku.np64(q), axis=-1, keepdims=True)
                                              * np.ones(D))[fits], "rows")
    assert np.isinf(ku.np64(got)[np.abs(want) > 3.42e38]).all()
    q[2, 1, 3], q[3, 0, 7] = float("inf"), float("nan")
    bad = rw4.qk_norm_rope(q, rotate=True)[0]
    assert not torch.isfinite(bad[2, 1]).any() and torch.isnan(bad[3, 0]).all()
    bad[2, 1], bad[3, 0] = got[2, 1], got[3, 0]
    assert torch.equal(bad, got)


def test_append_special_rows_under_a_norm():
    D = 128
    x = np.random.default_rng(36).standard_normal((5, 1, D)).astype(np.float32)
    x[1, 0, 3], x[2, 0, 9], x[3] = np.inf, np.nan, 0
    t, w = ku.dev(x), torch.ones(D, device=ku.DEV)
    for rotate in (False, True):
        cache = rw4.KVCache.empty(1, 16, 1, D)
        rw4.kv_append(cache, t, t, torch.arange(5, device=ku.DEV), k_weight=w, rotate=rotate)
        codes, scale = ku.opened(cache.k)[0, 0], cache.k_scale[0, 0].tolist()
        assert np.isnan(scale[1]) and np.isnan(scale[2]) and scale[3] == 0 and scale[0] > 0 and scale[4] > 0
        assert (codes[1:4] == 0).all() and (codes[[0, 4]] != 0).any(-1).all()


@pytest.mark.parametrize("D,dtype,B", [(64, BF16, 40), (128, BF16, 40), (128, F32, 90), (256, BF16, 40), (256, F32, 40)])
def test_attention_one_long_request_beside_many_short(D, dtype, B):
    # units enough for whole ones, but one request far longer than the others: its units are cut
    rng = np.random.default_rng(37)
    hk, group, page = 4, 8, 64
    q_lens = [40] + rng.integers(130, 200, B - 1).tolist()
    kv_lens = [9000] + q_lens[1:]
    if B > 64:
        q_lens[50], kv_lens[50] = 0, 7000  # a long request without queries
    pages = sum(-(-n // page) for n in kv_lens)
    table = ku.page_table(rng, kv_lens, page, -(-9000 // page), pages)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = ku.dev(rng.standard_normal((int(cu[-1]), hk * group, D)).astype(np.float32), dtype)
    td, kd, cd = ku.dev(table), ku.dev(np.array(kv_lens, np.int32)), ku.dev(cu)
    out, lse = rw4.kv_attention(q, cache, td, kd, cd, max_q_len=max(q_lens), return_lse=True)
    few, lse2 = rw4.kv_attention(q, cache, td, kd, cd, max_q_len=1, return_lse=True)  # the other kernel
    mags = rw4.kv_attention(q, ku.cache_of(ck, sk, np.abs(cv), sv), td, kd, cd, max_q_len=1, unrotate=False,
                            out_dtype=F32)
    reach = 1.01 * ku.np64(mags).sum(-1) / D ** 0.5
    size = D ** -0.5 * 7 * float(sk.max()) * ku.np64(q.float().abs().sum(-1))
    # both sides have the tolerance against the definition
    tol = 2 * ku.attention_tolerance(ku.np64(few), reach, size, dtype, D, 9000)
    ku.close(ku.np64(out), ku.np64(few), tol, "kernels")
    lt = 2 * ((D + 8) * ku.U24 * size + (64 + 4096) * ku.U24 + 4 * ku.U24 * np.abs(ku.np64(lse2)))
    ku.close(ku.np64(lse), ku.np64(lse2), lt, "lse")
    for b in (0, B - 1):
        rows = slice(int(cu[b]), int(cu[b]) + 6)
        want, wl, reach1, size1 = okv.kv_attention(ku.np64(q[rows]), ck, sk, cv, sv, pages, table[b:b + 1],
                                                   [kv_lens[b] - q_lens[b] + 6], [0, 6], D ** -0.5, True, 0, True)
        ku.close(ku.np64(out[rows]), want, ku.attention_tolerance(want, reach1, size1, dtype, D, kv_lens[b]), f"request {b}")


@pytest.mark.parametrize("new", [3, 4, 5000, 2 ** 31 - 1])
def test_slots_of_the_longest_requests(new):
    # requests end at 2^31 - 8192 tokens, what attention works on: more are refused, places stay in 32 bits
    page, width, most = 1 << 20, 4096, 2 ** 31 - 8192
    ctx = np.array([most - 3, 5, most - 2 ** 20], np.int32)
    add = np.array([new, 2, 1], np.int32)
    table = np.arange(3 * width, dtype=np.int32).reshape(3, width)
    ring, state = np.arange(20000, 20008, dtype=np.int32), np.array([3, 8], np.int32)
    tokens = min(new, 5000) + 5
    want = okv.kv_slots(ctx, add, table, ring, state, page, tokens) if new < 10 ** 6 else None
    d = [ku.dev(x) for x in (ctx, add, table, ring, state)]
    got = rw4.kv_slots(*d, page, tokens)
    torch.cuda.synchronize()
    assert got.served.tolist() == [int(new == 3), 1, 1]
    assert got.kv_len.tolist() == [most if new == 3 else most - 3, 7, most - 2 ** 20 + 1]
    if want is not None:
        have = [got.kv_len, got.cu_new, got.served, got.slot_map, got.positions, d[2], d[3], got.free_state]
        for x, y in zip(have, want):
            assert np.array_equal(x.cpu().numpy(), y)
    else:
        assert (got.slot_map == -1).all() and (got.positions == -1).all()


def test_append_of_more_tokens_than_a_grid_has_threads():
    # 2^26 + 70000 tokens, one key and value for all of them; all but a few store nothing
    D, T, page = 64, 2 ** 26 + 70000, 16
    rng = np.random.default_rng(38)
    x = ku.dev(rng.standard_normal((2, 1, D)).astype(np.float32), BF16)
    k, v = x[:1].expand(T, 1, D), x[1:].expand(T, 1, D)
    cache, small = rw4.KVCache.empty(2, page, 1, D), rw4.KVCache.empty(2, page, 1, D)
    slots = torch.full((T,), -1, dtype=torch.int64, device=ku.DEV)
    for s, t in enumerate((0, 2 ** 25 - 1, 2 ** 25, 2 ** 26, T - 1)):
        slots[t] = 5 * s
    rw4.kv_append(cache, k, v, slots)
    rw4.kv_append(small, k[:5], v[:5], torch.arange(5, device=ku.DEV) * 5)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, n), getattr(small, n)), n
    assert (cache.k_scale > 0).sum() == 5


def test_attention_of_more_units_than_a_grid_has_blocks():
    # 16400 requests of a token and 1024 heads each: 2^24 units and more in the kernel for many rows
    D, heads, page, B = 64, 1024, 16, 16400
    rng = np.random.default_rng(39)
    ck, sk = ku.pool(rng, 1, heads, page, D)
    cv, sv = ku.pool(rng, 1, heads, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    one = ku.dev(rng.standard_normal((1, heads, D)).astype(np.float32), BF16)
    lens = np.arange(B) % page + 1
    args = [ku.dev(np.zeros((B, 1), np.int32)), ku.dev(lens.astype(np.int32)), ku.dev(np.arange(B + 1, dtype=np.int32))]
    out = rw4.kv_attention(one.expand(B, heads, D), cache, *args, max_q_len=B)
    some = out[:page]
    assert torch.equal(out, some.repeat(B // page, 1, 1))
    q = ku.np64(one.expand(page, heads, D))[:, :8]
    want, _, reach, size = okv.kv_attention(q, ck[:, :8], sk[:, :8], cv[:, :8], sv[:, :8], 1, np.zeros((page, 1), np.int32),
                                            lens[:page], np.arange(page + 1), D ** -0.5, True, 0, True)
    ku.close(ku.np64(some)[:, :8], want, ku.attention_tolerance(want, reach, size, BF16, D, page), "out")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_lens,hint", [([1], 1), ([8], 8), ([1] * 40, 1), ([1] * 40, 40), ([70, 9, 200], 200),
                                         ([70, 9, 200], 1)])
def test_attention_stays_in_its_workspace(D, dtype, q_lens, hint):
    # cut units in a workspace of exactly the bytes asked for: what lies behind it stays
    rng = np.random.default_rng(40)
    hk, group, page, n = 2, 4, 64, 8000
    pages, B, T = n // page, len(q_lens), sum(q_lens)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    table = ku.dev(np.stack([rng.permutation(pages) for _ in range(B)]).astype(np.int32))
    lens = ku.dev((n - rng.integers(0, 500, B)).astype(np.int32))
    cu = ku.dev(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32))
    q = ku.dev(rng.standard_normal((T, hk * group, D)).astype(np.float32), dtype)
    nbytes = rw4.kv_attention_workspace_bytes(T, B, hk * group, hk, D)
    room = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device=ku.DEV)
    cache = ku.cache_of(ck, sk, cv, sv)
    got = rw4.kv_attention(q, cache, table, lens, cu, max_q_len=hint, workspace=room[:nbytes])
    assert (room[nbytes:] == 0xA5).all() and (room[:nbytes] != 0xA5).any()
    room.fill_(0xFF)  # and nothing in it is read before it is written
    assert torch.equal(rw4.kv_attention(q, cache, table, lens, cu, max_q_len=hint, workspace=room[:nbytes]), got)
    assert torch.isfinite(got).all() and (room[nbytes:] == 0xFF).all()
    with pytest.raises(ValueError, match="workspace"):
        rw4.kv_attention(q, cache, table, lens, cu, workspace=room[:nbytes - 16])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ratio", range(17, 24))
def test_attention_many_rows_first_row_of_a_small_value(D, ratio):
    # two keys, the first row sees the one with a value 2^ratio times smaller alone: 11 bits of it all the same
    rng = np.random.default_rng(41)
    page, heads, seeds = 16, 64, 40
    pages = seeds
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    sv[:, 0, 0] = 2.0 ** -ratio * rng.uniform(1, 2, seeds)
    sv[:, 0, 1] = rng.uniform(1, 2, seeds)
    q = ku.dev(rng.standard_normal((2 * seeds, heads, D)).astype(np.float32), BF16)
    table, lens, cu = np.arange(pages, dtype=np.int32)[:, None], np.full(seeds, 2, np.int32), 2 * np.arange(seeds + 1)
    out = ku.np64(rw4.kv_attention(q, ku.cache_of(ck, sk, cv, sv), ku.dev(table), ku.dev(lens),
                                   ku.dev(cu.astype(np.int32)), max_q_len=2, unrotate=False))[::2]
    want = (cv[:, 0, 0].astype(np.float64) * sv[:, 0, 0].astype(np.float64)[:, None])[:, None, :]
    tol = (2.0 ** -11 + 2 * ku.U24) * np.abs(want).max(-1, keepdims=True) + ku.half_step(BF16) * np.abs(want)
    ku.close(out, np.broadcast_to(want, out.shape), np.broadcast_to(tol, out.shape), "first rows")
