"""kv_attention's kernels in combinations of layout, type, mask and batch that
the tests of single features leave out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv as okv  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests import kv_util as ku  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
FULL = [(64, BF16), (128, BF16), (256, BF16), (64, F32), (128, F32), (256, F32)]


def _check(D, dtype, q_lens, kv_lens, group=4, hk=1, page=16, hint=None, layout="hnd", causal=True, window=0,
           unrotate=True, q_scale=1.8, out_dtype=None, pad=0, seed=50):
    """A call against the oracle: out, lse, and the rows of no request as they were."""
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // page) for n in kv_lens) + 1
    table = ku.page_table(rng, kv_lens, page, max(-(-n // page) for n in kv_lens) + 1, pages)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    cache = ku.cache_of(ck, sk, cv, sv, layout)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    n = int(cu[-1])
    q = ku.dev((q_scale * rng.standard_normal((n + pad, hk * group, D))).astype(np.float32), dtype)
    out_dtype = dtype if out_dtype is None else out_dtype
    out = torch.full((n + pad, hk * group, D), 7.0, dtype=out_dtype, device=ku.DEV)
    lse = torch.full((n + pad, hk * group), 7.0, device=ku.DEV)
    rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array(kv_lens, np.int32)), ku.dev(cu),
                     max_q_len=max(q_lens) if hint is None else hint, causal=causal, window=window, unrotate=unrotate,
                     out=out, lse=lse)
    want, wl, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, kv_lens, cu, D ** -0.5, causal,
                                             window, unrotate)
    most = max(kv_lens)
    tol = ku.attention_tolerance(want[:n], reach[:n], size[:n], out_dtype, D, most)
    ku.close(ku.np64(out)[:n], want[:n], tol, "out")
    seen = np.where(np.isfinite(wl[:n]), wl[:n], 0)
    lt = (D + 8) * ku.U24 * size[:n] + (64 + min(most, 4096)) * ku.U24 + 4 * ku.U24 * np.abs(seen)
    ku.close(ku.np64(lse)[:n], wl[:n], lt, "lse")
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()


# rows of a request pass the kernel for few rows in all of these (group 4, 70 tokens)
WIDE = {
    "plain": {},
    "slots_outside": dict(layout="nhd", hk=2, group=2, q_lens=[40, 70]),
    "sharp": dict(q_scale=30.0),
    "window": dict(window=37),
    "window_beyond": dict(window=10 ** 12),
    "cross": dict(causal=False),
    "plain_domain": dict(unrotate=False),
    "padding": dict(pad=150),
    "group_3": dict(group=3),
    "group_64": dict(group=64, q_lens=[3, 5]),
    "more_rows_than_keys": dict(kv_lens=[30, 9]),
}


@pytest.mark.parametrize("D,dtype", FULL)
@pytest.mark.parametrize("name", WIDE)
def test_many_rows(name, D, dtype):
    _check(D, dtype, **{"q_lens": [70, 66], "kv_lens": [301, 66], **WIDE[name]})


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, BF16)])
def test_many_rows_of_mixed_types(D, dtype, out_dtype):
    _check(D, dtype, [70, 66], [301, 66], out_dtype=out_dtype)


@pytest.mark.parametrize("D,dtype", FULL)
@pytest.mark.parametrize("hint", [1, 10 ** 6])
def test_more_requests_than_threads(D, dtype, hint):
    # 300 and 1030 requests: several for each of a block's threads; some without tokens, some without keys
    rng = np.random.default_rng(51)
    for B in (300, 1030):
        q_lens, kv_lens = rng.integers(0, 3, B), rng.integers(0, 40, B)
        q_lens[0], q_lens[B - 1], kv_lens[B - 1] = 0, 2, 40
        _check(D, dtype, q_lens.tolist(), kv_lens.tolist(), group=2, hint=hint, seed=B)


@pytest.mark.parametrize("D,dtype", FULL)
def test_single_tokens_and_chunks_in_one_call(D, dtype):
    # a serving step: decoding requests beside a prompt's chunk, with and without the hint
    q_lens, kv_lens = [1] * 9 + [90] + [1] * 9, list(range(5, 200, 22)) + [250] + list(range(7, 202, 22))
    for hint in (90, 10 ** 6, 1):
        _check(D, dtype, q_lens, kv_lens, hint=hint, pad=5)


@pytest.mark.parametrize("D,dtype", FULL)
@pytest.mark.parametrize("hint", [1, 80])
def test_starts_out_of_range_leave_other_rows(D, dtype, hint):
    # starts below 0, beyond the tokens or falling: clamped, and rows of no request stay as they were
    rng = np.random.default_rng(52)
    page, pages, T = 16, 12, 80
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = rng.permutation(pages).reshape(2, 6).astype(np.int32)
    q = ku.dev(rng.standard_normal((T, 2, D)).astype(np.float32), dtype)

    def run(cu, kv):
        out = torch.full_like(q, 5.0)
        rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array(kv, np.int32)), ku.dev(np.array(cu, np.int32)),
                         max_q_len=hint, out=out)
        return ku.np64(out)

    def want(cu, kv):
        w, _, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, kv, cu, D ** -0.5, True, 0, True)
        return w, ku.attention_tolerance(w, reach, size, dtype, D, 96)

    got = run([-7, -7, 1000], [-4, 90])  # no tokens; all of them
    w, tol = want([0, 0, T], [0, 90])
    ku.close(got, w, tol, "second request")
    got = run([2 ** 31 - 1, 5, -2 ** 31], [50, 90])  # falling: nobody has any
    assert (got == 5.0).all()
    got = run([60, 20, 33], [50, 96])  # the first falls, the second is rows 20..32
    w, tol = want([20, 20, 33], [50, 96])
    ku.close(got[20:33], w[20:33], tol[20:33], "rows of the second")
    assert (got[:20] == 5.0).all() and (got[33:] == 5.0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [3, 40])
def test_bad_pages_under_both_kernels(D, rows):
    # pages out of range and a length beyond the table, fp32, with few and with many rows
    rng = np.random.default_rng(53)
    page, pages = 16, 12
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = np.array([[0, -1, 2, 12, 4, 5], [6, 7, 8, 9, 2 ** 31 - 1, -2 ** 31]], np.int32)
    cu, lens = [0, rows, 2 * rows], [75, 10 ** 9]
    q = ku.dev(rng.standard_normal((2 * rows, 4, D)).astype(np.float32))
    out = rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array(lens, np.int32)), ku.dev(np.array(cu, np.int32)),
                           max_q_len=rows)
    w, _, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, [75, 96], cu, D ** -0.5, True, 0, True)
    ku.close(ku.np64(out), w, ku.attention_tolerance(w, reach, size, F32, D, 96), "out")


@pytest.mark.parametrize("D,dtype", [(256, F32), (256, BF16), (64, F32)])
def test_captured_many_rows_replay(D, dtype):
    # instances of the kernel for many rows under capture; lengths and value scales change between replays
    rng = np.random.default_rng(54)
    page = 16
    ck, sk = ku.pool(rng, 80, 2, page, D)
    cv, sv = ku.pool(rng, 80, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = ku.dev(rng.permutation(80).reshape(2, 40).astype(np.int32))
    kv, cu = ku.dev(np.array([500, 640], np.int32)), ku.dev(np.array([0, 70, 150], np.int32))
    q = ku.dev(rng.standard_normal((150, 8, D)).astype(np.float32), dtype)
    out = torch.zeros_like(q)
    call = rw4.prepare_kv_attention(q, cache, table, kv, cu, max_q_len=80, out=out)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    scales = cache.v_scale.clone()
    for n, lens in enumerate(([500, 640], [90, 80], [640, 81], [1, 333])):
        kv.copy_(ku.dev(np.array(lens, np.int32)))
        cache.v_scale.copy_(scales * (1e-7 if n % 2 else 1.0))
        cache.v_scale[::3] *= 1e6 if n == 3 else 1.0
        out.fill_(9.0)
        g.replay()
        junk = torch.randn(1000, device=ku.DEV).sum()
        torch.cuda.synchronize()
        want = rw4.kv_attention(q, cache, table, kv, cu, max_q_len=80)
        assert torch.equal(out, want) and torch.isfinite(junk) and torch.isfinite(out).all()
