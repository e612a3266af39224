"""kv_attention with a window and sinks (first keys that stay visible) against the
oracle: both kernels, cut and whole units, sinks before, at and beyond the window's
start, keys between sinks and window poisoned, captured steps whose lengths move."""
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


def _poison(sk, sv, table, kv_lens, q_lens, page, window, sinks):
    """NaN scales in every slot that no row of its request may see."""
    see = np.zeros(sk.shape[0] * page, bool)
    for b, (n, q) in enumerate(zip(kv_lens, q_lens)):
        j = np.arange(n)
        visible = (j < sinks) | (j > n - q - window)  # of the first row, or of a later one
        see[table[b, j[visible] // page] * page + j[visible] % page] = True
    hidden = ~see.reshape(sk.shape[0], 1, page)
    return np.where(hidden, np.float32("nan"), sk), np.where(hidden, np.float32("inf"), sv)


def _check(D, dtype, q_lens, kv_lens, window, sinks, group=4, hk=1, page=16, hint=None, unrotate=True, out_dtype=None,
           pad=0, poison=True, layout="hnd", seed=60):
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // page) for n in kv_lens) + 1
    table = ku.page_table(rng, kv_lens, page, max(-(-n // page) for n in kv_lens) + 1, pages)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    if poison:
        pk, pv = _poison(sk, sv, table, kv_lens, q_lens, page, window, sinks)
        cache = ku.cache_of(ck, pk, cv, pv, layout)
    else:
        cache = ku.cache_of(ck, sk, cv, sv, layout)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    n = int(cu[-1])
    q = ku.dev((1.8 * rng.standard_normal((n + pad, hk * group, D))).astype(np.float32), dtype)
    out_dtype = dtype if out_dtype is None else out_dtype
    out = torch.full((n + pad, hk * group, D), 7.0, dtype=out_dtype, device=ku.DEV)
    lse = torch.full((n + pad, hk * group), 7.0, device=ku.DEV)
    rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array(kv_lens, np.int32)), ku.dev(cu),
                     max_q_len=max(q_lens) if hint is None else hint, window=window, sinks=sinks, unrotate=unrotate,
                     out=out, lse=lse)
    want, wl, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, kv_lens, cu, D ** -0.5, True,
                                             window, unrotate, sinks)
    most = min(max(kv_lens), window + sinks)
    tol = ku.attention_tolerance(want[:n], reach[:n], size[:n], out_dtype, D, most)
    ku.close(ku.np64(out)[:n], want[:n], tol, "out")
    seen = np.where(np.isfinite(wl[:n]), wl[:n], 0)
    lt = (D + 8) * ku.U24 * size[:n] + (64 + min(most, 4096)) * ku.U24 + 4 * ku.U24 * np.abs(seen)
    ku.close(ku.np64(lse)[:n], wl[:n], lt, "lse")
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()


# sinks: one, within a step, a whole step, one more, several steps, all of the request
SINKS = [1, 4, 63, 64, 65, 200, 10 ** 12]


@pytest.mark.parametrize("D,dtype", FULL)
@pytest.mark.parametrize("sinks", SINKS)
def test_few_rows(sinks, D, dtype):
    _check(D, dtype, [1, 3, 2, 1, 1], [700, 333, 40, 1, 129], 100, sinks)


@pytest.mark.parametrize("D,dtype", FULL)
@pytest.mark.parametrize("sinks", SINKS)
def test_many_rows(sinks, D, dtype):
    _check(D, dtype, [70, 66, 33], [701, 66, 400], 90, sinks)


@pytest.mark.parametrize("D,dtype", [(64, F32), (128, BF16), (256, BF16)])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 500, 10 ** 12])
@pytest.mark.parametrize("rows", [1, 70])
def test_windows(window, rows, D, dtype):
    _check(D, dtype, [rows, rows], [650, 128 + rows], window, 5)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (128, F32), (256, F32)])
@pytest.mark.parametrize("name,kw", [
    ("cut_units", dict(q_lens=[1, 2], kv_lens=[6000, 9001], window=5000, sinks=300)),
    ("cut_chunk", dict(q_lens=[150], kv_lens=[4000], window=3000, sinks=130)),
    ("prompt_past_its_window", dict(q_lens=[400, 333], kv_lens=[400, 333], window=70, sinks=20)),
    ("chunk_past_its_window", dict(q_lens=[300], kv_lens=[900], window=50, sinks=66, hk=2, group=2)),
    ("more_rows_than_keys", dict(q_lens=[70, 20], kv_lens=[30, 9], window=8, sinks=3)),
    ("hint_too_small", dict(q_lens=[90, 70], kv_lens=[500, 300], window=40, sinks=70, hint=1)),
    ("hint_too_large", dict(q_lens=[1, 1], kv_lens=[500, 300], window=40, sinks=70, hint=1000)),
    ("slots_outside", dict(q_lens=[3, 70], kv_lens=[300, 500], window=64, sinks=64, layout="nhd", hk=2, group=3)),
    ("plain_domain", dict(q_lens=[2, 1], kv_lens=[300, 500], window=64, sinks=9, unrotate=False)),
    ("padding", dict(q_lens=[2, 1], kv_lens=[300, 500], window=64, sinks=9, pad=90)),
    ("large_pages", dict(q_lens=[1, 65], kv_lens=[700, 900], window=128, sinks=130, page=256)),
    ("no_keys", dict(q_lens=[1, 2, 1], kv_lens=[0, 300, 0], window=16, sinks=2)),
], ids=lambda x: x if isinstance(x, str) else "")
def test_shapes(name, kw, D, dtype):
    _check(D, dtype, **kw)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("rows", [1, 70])
def test_mixed_types(rows, dtype, out_dtype):
    _check(128, dtype, [rows], [400], 60, 17, out_dtype=out_dtype)


@pytest.mark.parametrize("hint", [1, 200])
def test_many_requests(hint):
    rng = np.random.default_rng(3)
    kv = [int(x) for x in rng.integers(0, 400, 300)]
    _check(64, BF16, [1] * 300, kv, 50, 30, hint=hint)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, F32)])
@pytest.mark.parametrize("name,kv,window", [("even", 700, 300), ("ragged", None, 500), ("long_beside_short", -1, 4000)])
def test_whole_and_cut_units_of_few_rows(name, kv, window, D, dtype):
    # 70 requests of 4 KV heads: 280 units, each a block's (even, ragged), or cut (one request of 30 times the others' keys)
    rng = np.random.default_rng(8)
    kv = [kv] * 70 if kv and kv > 0 else [int(x) for x in rng.integers(1, 700 if kv is None else 130, 70)]
    if name == "long_beside_short":
        kv[33] = 3900
    _check(D, dtype, [1 + i % 2 for i in range(70)], kv, window, 21, hk=4, group=2)


def test_a_sink_on_a_bad_page_is_hidden():
    rng = np.random.default_rng(4)
    page, D = 16, 128
    table = np.arange(40, dtype=np.int32)[None].copy()
    table[0, 1] = 999   # keys 16..31 have no page
    ck, sk = ku.pool(rng, 40, 1, page, D)
    cv, sv = ku.pool(rng, 40, 1, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    for rows in (1, 70):
        q = ku.dev(rng.standard_normal((rows, 4, D)).astype(np.float32), F32)
        cu = np.array([0, rows], np.int32)
        out = rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array([600], np.int32)), ku.dev(cu), max_q_len=rows,
                               window=90, sinks=40)
        want, _, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, 40, table, [600], cu, D ** -0.5, True, 90,
                                                True, 40)
        ku.close(ku.np64(out), want, ku.attention_tolerance(want, reach, size, F32, D, 130), f"{rows} rows")


def test_without_effect():
    # no window, no sinks, or all of a request: the plain call's bits where the same kernels run
    rng = np.random.default_rng(5)
    page, D, kv = 16, 128, 333
    table = np.arange(24, dtype=np.int32)[None]
    cache = ku.cache_of(*ku.pool(rng, 24, 2, page, D), *ku.pool(rng, 24, 2, page, D))
    q = ku.dev(rng.standard_normal((3, 8, D)).astype(np.float32), BF16)
    args = (q, cache, ku.dev(table), ku.dev(np.array([kv], np.int32)), ku.dev(np.array([0, 3], np.int32)))
    plain = rw4.kv_attention(*args, max_q_len=3)
    assert torch.equal(rw4.kv_attention(*args, max_q_len=3, sinks=7), plain)
    windowed = rw4.kv_attention(*args, max_q_len=3, window=50)
    assert torch.equal(rw4.kv_attention(*args, max_q_len=3, window=50, sinks=0), windowed)
    assert not torch.equal(rw4.kv_attention(*args, max_q_len=3, window=50, sinks=1), windowed)


def test_one_long_request():
    # 2^31 - 8192 tokens, all on one page
    D, page = 64, 1 << 20
    rng = np.random.default_rng(6)
    few = 4096  # rows that repeat over the page
    cache = rw4.KVCache.empty(1, page, 1, D, ku.DEV)
    ck, sk = ku.pool(rng, 1, 1, few, D)
    cv, sv = ku.pool(rng, 1, 1, few, D)
    for to, x in ((cache.k, ku.stored(ck)), (cache.v, ku.stored(cv)), (cache.k_scale, sk), (cache.v_scale, sv)):
        to.view(page // few, *x.shape[2:]).copy_(ku.dev(x[0]))
    width = 2048
    n = 2 ** 31 - 8192
    table = torch.zeros(1, width, dtype=torch.int32, device=ku.DEV)
    q = ku.dev(rng.standard_normal((2, 4, D)).astype(np.float32), F32)
    cu = ku.dev(np.array([0, 2], np.int32))
    for hint in (2, 1000):
        got = rw4.kv_attention(q, cache, table, ku.dev(np.array([2 ** 31 - 1], np.int32)), cu, max_q_len=hint, window=70,
                               sinks=5)
        for t in range(2):
            place = n - 2 + t
            j = np.concatenate([np.arange(5), np.arange(place - 69, place + 1)])
            at = j % few
            kc, vc = ck[:, :, at], cv[:, :, at]
            s, v = sk[:, :, at], sv[:, :, at]
            want, _, reach, size = okv.kv_attention(ku.np64(q)[t:t + 1], kc, s, vc, v, 1, np.zeros((1, 1), np.int32),
                                                    [len(j)], [0, 1], D ** -0.5, False, 0, True)
            ku.close(ku.np64(got)[t:t + 1], want, ku.attention_tolerance(want, reach, size, F32, D, 75), f"row {t}")


def test_captured_steps_follow_their_lengths():
    rng = np.random.default_rng(7)
    page, D, B = 16, 128, 3
    table = np.arange(3 * 60, dtype=np.int32).reshape(3, 60)
    ck, sk = ku.pool(rng, 180, 2, page, D)
    cv, sv = ku.pool(rng, 180, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    q = ku.dev(rng.standard_normal((B, 8, D)).astype(np.float32), BF16)
    kv_len, cu = torch.zeros(B, dtype=torch.int32, device=ku.DEV), ku.dev(np.arange(B + 1, dtype=np.int32))
    out = torch.empty_like(q)
    call = rw4.prepare_kv_attention(q, cache, ku.dev(table), kv_len, cu, max_q_len=1, window=100, sinks=70, out=out)
    kv_len.fill_(500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([500, 1, 960], [64, 171, 170], [0, 134, 135], [800, 801, 802]):
        kv_len.copy_(ku.dev(np.array(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = rw4.kv_attention(q, cache, ku.dev(table), kv_len, cu, max_q_len=1, window=100, sinks=70)
        assert torch.equal(got, want), lens
        ref, _, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, 180, table, lens, np.arange(B + 1), D ** -0.5,
                                               True, 100, True, 70)
        ku.close(ku.np64(got), ref, ku.attention_tolerance(ref, reach, size, BF16, D, 170), str(lens))


def test_refusals():
    cache = rw4.KVCache.empty(2, 16, 1, 128, ku.DEV)
    q = torch.zeros(1, 1, 128, device=ku.DEV)
    i32 = dict(dtype=torch.int32, device=ku.DEV)
    args = (q, cache, torch.zeros(1, 2, **i32), torch.ones(1, **i32), torch.tensor([0, 1], **i32))
    with pytest.raises(rw4.RW4Error, match="SHAPE"):
        rw4.kv_attention(*args, window=8, sinks=-1)
    with pytest.raises(rw4.RW4Error, match="UNSUPPORTED"):
        rw4.kv_attention(*args, window=8, sinks=1, causal=False)
