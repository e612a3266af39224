"""The INT4 KV cache's serving operators against the float64 oracle: slots,
head norms with rotary positions, append, attention, and a run of them."""
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


# ---------------------------------------------------------------- slots
def _slots_case(seed, B, page, new_max, ctx_max, finished, short, tokens=None, wide=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_max + 1, B)
    new = rng.integers(0, new_max + 1, B)
    new[rng.permutation(B)[:finished]] = -1
    width = -(-(ctx_max + new_max) // page) + 1 - wide
    have = -(-ctx // page)
    cap = int(have.sum()) + B * (new_max // page + 2) + 1
    ids = rng.permutation(cap)
    table = np.full((B, max(width, 1)), -1, np.int32)
    at = 0
    for b in range(B):
        n = min(have[b], table.shape[1])
        table[b, :n] = ids[at:at + n]
        at += n
    need = np.where(new >= 0, -(-(ctx + np.maximum(new, 0)) // page) - have, 0)
    count = max(0, int(need.sum()) - short) if short else cap - at
    ring = np.full(cap, -1, np.int32)
    head = int(rng.integers(0, cap))
    ring[(head + np.arange(cap - at)) % cap] = ids[at:]
    total = int(np.maximum(new, 0).sum())
    return (ctx.astype(np.int32), new.astype(np.int32), table, ring, np.array([head, count], np.int32), page,
            total + 5 if tokens is None else tokens)


SLOT_CASES = [
    # seed, B, page, new_max, ctx_max, finished, short, tokens, table columns too few
    (0, 1, 16, 1, 40, 0, 0, None, 0), (1, 1, 16, 500, 0, 0, 0, None, 0), (2, 7, 1, 3, 9, 2, 3, None, 0),
    (3, 64, 16, 1, 4000, 5, 0, None, 0), (4, 64, 16, 1, 4000, 5, 2, None, 0), (5, 257, 32, 90, 700, 40, 30, None, 0),
    (6, 300, 64, 400, 900, 60, 0, None, 2), (7, 4096, 16, 20, 300, 500, 900, None, 0), (8, 33, 128, 0, 500, 0, 0, 64, 0),
    (9, 12, 16, 50, 100, 1, 0, 40, 0), (10, 5, 16, 3, 20, 5, 0, 0, 0),
]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("case", SLOT_CASES, ids=[f"B{c[1]}_p{c[2]}_s{c[0]}" for c in SLOT_CASES])
def test_slots_match_oracle(case, alias):
    ctx, new, table, ring, state, page, tokens = _slots_case(*case)
    want = okv.kv_slots(ctx, new, table, ring, state, page, tokens)
    d = [ku.dev(x) for x in (ctx, new, table, ring, state)]
    out = dict(kv_len=d[0], free_state_out=d[4]) if alias else {}
    got = rw4.kv_slots(*d, page, tokens, **out)
    have = [got.kv_len, got.cu_new, got.served, got.slot_map, got.positions, d[2], d[3], got.free_state]
    names = "kv_len cu_new served slot_map positions table ring state".split()
    torch.cuda.synchronize()
    for name, x, y in zip(names, have, want):
        assert np.array_equal(x.cpu().numpy(), y), name


def test_slots_bad_device_values_stay_in_bounds():
    # negative lengths, a state outside the ring, pages of -1: nothing out of bounds, clamped results
    ctx = ku.dev(np.array([-5, 20, 2 ** 31 - 1], np.int32))
    new = ku.dev(np.array([3, 4, 2 ** 31 - 1], np.int32))
    table = ku.dev(np.full((3, 4), -1, np.int32))
    ring = ku.dev(np.arange(8, dtype=np.int32))
    got = rw4.kv_slots(ctx, new, table, ring, ku.dev(np.array([-3, 99], np.int32)), 16, 64)
    torch.cuda.synchronize()
    assert got.served.tolist() == [1, 1, 0]
    assert got.kv_len.tolist() == [3, 24, 2 ** 31 - 1]
    assert got.slot_map[:3].tolist() == [5 * 16, 5 * 16 + 1, 5 * 16 + 2]  # head -3 is entry 5 of 8
    assert got.slot_map[3:].tolist() == [-1] * 61  # request 1's page is -1, request 2 is refused
    assert got.free_state.tolist() == [6, 7]


# ---------------------------------------------------------------- head norms and rotary positions
def _rows(seed, T, heads, D, dtype, pad=0, big=1.0):
    """A [T, heads, D] view of a wider buffer, and its values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, heads + pad, D)) * np.exp(0.5 * rng.standard_normal((T, heads + pad, 1))) * big
    t = ku.dev(x.astype(np.float32), dtype)
    return t[:, pad // 2:pad // 2 + heads]


ROW_CASES = [
    # T, heads, kv heads, D, rot, interleaved, norm, dtype
    (1, 1, 1, 128, 128, False, True, BF16), (5, 32, 8, 128, 128, False, True, BF16),
    (33, 3, 1, 128, 64, True, True, F32), (7, 5, 5, 64, 64, False, True, BF16), (18, 9, 3, 64, 32, True, False, F32),
    (11, 4, 2, 256, 256, False, True, F32), (6, 7, 1, 256, 16, True, True, BF16), (9, 2, 2, 128, 0, False, True, F32),
    (13, 6, 2, 128, 96, False, False, BF16), (3000, 6, 2, 64, 64, True, True, BF16), (2100, 9, 3, 128, 128, False, True, F32),
]


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("case", ROW_CASES, ids=[f"T{c[0]}_h{c[1]}_{c[2]}_D{c[3]}_r{c[4]}" for c in ROW_CASES])
def test_norm_rope_matches_oracle(case, rotate):
    T, hq, hk, D, rot, inter, norm, dtype = case
    rng = np.random.default_rng(T)
    q, k = _rows(1, T, hq, D, dtype, pad=2), _rows(2, T, hk, D, dtype, pad=3)
    w = (1 + 0.3 * rng.standard_normal((2, D))).astype(np.float32) if norm else (None, None)
    cs = rw4.rope_table(700, rot) if rot else None
    pos = rng.integers(0, 700, T).astype(np.int32)
    wd = [None if x is None else ku.dev(x) for x in w]
    got = rw4.qk_norm_rope(q, k, wd[0], wd[1], cs, ku.dev(pos), interleaved=inter, rotate=rotate)
    for x, y, wt, name in ((q, got[0], w[0], "q"), (k, got[1], w[1], "k")):
        z, f = okv.norm_rope(ku.np64(x), wt, 1e-6, None if cs is None else ku.np64(cs), pos, inter)
        z = z * f
        want = okv.rotate_heads(z) if rotate else z
        # per row: the norm's sums (14 roundings, halved by the root), root and division (5), two products, the
        # rotary terms (3 sqrt 2), eight butterfly additions and the final product, each 2^-24 of the row's length
        tol = 32 * ku.U24 * np.linalg.norm(z, axis=-1, keepdims=True) + ku.half_step(dtype) * np.abs(want)
        ku.close(ku.np64(y), want, tol, name)
        assert y.dtype is dtype


def test_norm_rope_in_place_skips_padding_and_queries_alone():
    T, D = 21, 128
    q, k = _rows(3, T, 4, D, BF16, pad=1), _rows(4, T, 2, D, BF16, pad=1)
    w = torch.ones(D, device=ku.DEV)
    cs = rw4.rope_table(64, D)
    pos = ku.dev(np.arange(T, dtype=np.int32))
    pos[5], pos[6], pos[20] = -1, 64, -2 ** 31
    want = rw4.qk_norm_rope(q, k, w, w, cs, pos.clamp(0, 63))
    alone = rw4.qk_norm_rope(q, None, w, None, cs, pos.clamp(0, 63))
    assert alone[1] is None and torch.equal(alone[0], want[0])
    q0, k0 = q.clone(), k.clone()
    got = rw4.qk_norm_rope(q, k, w, w, cs, pos, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    for t in range(T):
        keep = t in (5, 6, 20)
        assert torch.equal(q[t], q0[t] if keep else want[0][t]) and torch.equal(k[t], k0[t] if keep else want[1][t])
    mixed = rw4.qk_norm_rope(q0, k0, w, w, cs, pos.clamp(0, 63), out_dtype=F32)
    assert mixed[0].dtype is F32 and torch.equal(mixed[0].to(BF16), want[0])


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("case", ROW_CASES, ids=[f"T{c[0]}_h{c[1]}_{c[2]}_D{c[3]}_r{c[4]}" for c in ROW_CASES])
def test_append_matches_oracle(case, rotate, layout):
    T, hq, hk, D, rot, inter, norm, dtype = case
    page = 16 if T < 30 else 64
    pages = -(-T // page) + 1
    rng = np.random.default_rng(T + 1)
    q, k, v = _rows(1, T, hq, D, dtype, pad=1), _rows(2, T, hk, D, dtype, pad=3), _rows(5, T, hk, D, dtype, pad=2)
    w = (1 + 0.3 * rng.standard_normal((2, D))).astype(np.float32) if norm else (None, None)
    wd = [None if x is None else ku.dev(x) for x in w]
    cs = rw4.rope_table(700, rot) if rot else None
    pos = rng.integers(0, 700, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    old = [ku.pool(rng, pages, hk, page, D) for _ in range(2)]
    cache = ku.cache_of(*old[0], *old[1], layout)
    dense = rw4.qk_norm_rope(q, None, wd[0], None, cs, ku.dev(pos), interleaved=inter, rotate=rotate)[0]
    got = rw4.kv_append(cache, k, v, ku.dev(slots), q, wd[0], wd[1], cs, ku.dev(pos), interleaved=inter, rotate=rotate)
    assert torch.equal(got, dense)
    csn = None if cs is None else ku.np64(cs)
    zk, fk = okv.norm_rope(ku.np64(k), w[1], 1e-6, csn, pos, inter)
    zv, fv = ku.np64(v), np.ones((T, hk, 1))
    for z, f, (codes, scales), packed, sc, name in ((zk, fk, old[0], cache.k, cache.k_scale, "k"),
                                                    (zv, fv, old[1], cache.v, cache.v_scale, "v")):
        c, s = okv.quantize_heads(z, f, rotate)
        want_c, want_s = codes.copy(), scales.astype(np.float64)
        want_c[slots // page, :, slots % page] = c
        want_s[slots // page, :, slots % page] = s
        assert np.array_equal(ku.opened(packed), want_c), name  # rows behind the slots as they were
        # fp32: the maximum, 1 / 7, 1 / sqrt(D) and their products (6 roundings), the norm's factor (its sum, 14
        # roundings halved by the root, root and division, 5)
        ku.close(ku.np64(sc), want_s, np.abs(want_s) * 18 * ku.U24, name + " scale")


def test_append_ties_zeros_and_special_rows():
    D = 128
    cache = rw4.KVCache.empty(2, 16, 1, D)
    x = np.zeros((6, 1, D), np.float32)
    x[1, 0] = 0.5 * np.arange(D) % 7 - 3.0
    x[1, 0, 0] = 7.0  # m = 7: the codes are x itself, halves are exact ties
    x[2, 0, 3] = np.inf
    x[3, 0, 9] = np.nan
    x[4, 0, :2] = 1e-38, -1e-38
    x[5, 0, :2] = 3e38, 3e38
    t = ku.dev(x)
    slots = ku.dev(np.array([0, 1, 2, 3, 20, 31], np.int64))
    rw4.kv_append(cache, t, t, slots, rotate=False)
    codes, scale = ku.opened(cache.k), cache.k_scale.cpu().numpy()
    assert (codes[0, 0, 0] == 0).all() and scale[0, 0, 0] == 0
    assert np.array_equal(codes[0, 0, 1], np.rint(x[1, 0].astype(np.float64)))
    for i in (2, 3):
        assert (codes[0, 0, i] == 0).all() and np.isnan(scale[0, 0, i])
    assert codes[1, 0, 4, :2].tolist() == [7, -7] and codes[1, 0, 15, :2].tolist() == [7, 7]
    assert torch.equal(cache.k, cache.v) and np.array_equal(scale, cache.v_scale.cpu().numpy(), equal_nan=True)
    rw4.kv_append(cache, t, t, slots)  # rotated: sums of 3e38 stay finite in fp64
    assert np.isfinite(cache.k_scale[1, 0, 15].item()) and (ku.opened(cache.k)[1, 0, 15, ::2] == 7).all()
    assert np.isnan(cache.k_scale[0, 0, 2].item()) and np.isnan(cache.v_scale[0, 0, 3].item())


def test_append_skips_slots_and_positions_out_of_range():
    D, T = 64, 8
    rng = np.random.default_rng(0)
    old = [ku.pool(rng, 2, 2, 16, D) for _ in range(2)]
    cache = ku.cache_of(*old[0], *old[1])
    k, v, q = _rows(1, T, 2, D, BF16), _rows(2, T, 2, D, BF16), _rows(3, T, 4, D, BF16)
    slots = np.array([0, -1, 32, 2 ** 40, -2 ** 60, 5, 6, 31], np.int64)
    pos = np.array([0, 1, 2, 3, 4, -1, 10, 9], np.int32)
    q_out = torch.full_like(q, 3.0)
    rw4.kv_append(cache, k, v, ku.dev(slots), q, cos_sin=rw4.rope_table(10, D), positions=ku.dev(pos), q_out=q_out)
    codes = ku.opened(cache.k)
    changed = np.argwhere((codes != old[0][0]).any(-1).any(1))
    assert changed.tolist() == [[0, 0], [1, 15]]  # slots 0 and 31; 5 and 6 have positions out of range
    assert (q_out[5:7] == 3.0).all() and not (q_out[[0, 1, 2, 3, 4, 7]] == 3.0).all(-1).any()


# ---------------------------------------------------------------- attention
def _attend(seed, q_lens, kv_lens, hq, hk, D, page, dtype, causal=True, window=0, unrotate=True, out_dtype=None,
            layout="hnd", scale=None, pad_rows=0, hint=True, q_scale=1.8):
    rng = np.random.default_rng(seed)
    out_dtype = dtype if out_dtype is None else out_dtype
    pages = sum(-(-n // page) for n in kv_lens) + 2
    width = max([-(-n // page) for n in kv_lens] + [0]) + 1
    table = ku.page_table(rng, kv_lens, page, width, pages)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(cu[-1]) + pad_rows
    q = (q_scale * rng.standard_normal((T, hq, D))).astype(np.float32)
    # what no row may see is poisoned: slots behind the lengths, pages of nobody
    bad_s, bad_v = np.full_like(sk, np.nan), np.full_like(sv, np.inf)
    for b, n in enumerate(kv_lens):
        for j in range(0, n, page):
            m = min(page, n - j)
            bad_s[table[b, j // page], :, :m] = sk[table[b, j // page], :, :m]
            bad_v[table[b, j // page], :, :m] = sv[table[b, j // page], :, :m]
    cache = ku.cache_of(ck, bad_s, cv, bad_v, layout)
    qd = ku.dev(q, dtype)
    out = torch.full((T, hq, D), 7.0, dtype=out_dtype, device=ku.DEV)
    lse = torch.full((T, hq), 7.0, device=ku.DEV)
    kv = ku.dev(np.array(kv_lens, np.int32))
    sc = D ** -0.5 if scale is None else scale
    rw4.kv_attention(qd, cache, ku.dev(table), kv, ku.dev(cu), max_q_len=max(q_lens) if hint else None, causal=causal,
                     window=window, unrotate=unrotate, out=out, lse=lse, scale=scale)
    want, wl, reach, size = okv.kv_attention(ku.np64(qd), ck, sk, cv, sv, pages, table, kv_lens, cu, sc, causal, window,
                                             unrotate)
    n = int(cu[-1])
    tol = ku.attention_tolerance(want[:n], reach[:n], size[:n], out_dtype, D, max(kv_lens + [1]))
    ku.close(ku.np64(out)[:n], want[:n], tol, "out")
    # the score's error, the sum's and the logarithm's
    lt = ((D + 8) * ku.U24 * size[:n] + 64 * ku.U24 + 4 * ku.U24 * np.abs(np.where(np.isfinite(wl[:n]), wl[:n], 0))
          + min(max(kv_lens + [1]), 4096) * ku.U24)
    ku.close(ku.np64(lse)[:n], wl[:n], lt, "lse")
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()  # rows of no request
    return out


ATT_CASES = {
    "one_key": ([1], [1], 1, 1, 128, 16, BF16, {}),
    "no_keys": ([1, 1], [0, 5], 4, 2, 128, 16, BF16, {}),
    "no_queries": ([0, 2, 0], [40, 33, 0], 4, 2, 64, 16, F32, {}),
    "decode": ([1] * 5, [1, 15, 16, 17, 300], 32, 8, 128, 16, BF16, {}),
    "decode_long": ([1], [5000], 8, 2, 128, 64, BF16, {}),
    "decode_f32": ([1, 1, 1], [700, 31, 64], 6, 2, 128, 32, F32, {}),
    "decode_64": ([1, 1, 1], [513, 40, 1], 14, 2, 64, 16, BF16, {}),
    "decode_256": ([1, 1], [513, 95], 5, 1, 256, 16, BF16, {}),
    "decode_256_f32": ([1, 1], [130, 95], 4, 1, 256, 128, F32, {}),
    "decode_group_16": ([1, 1], [200, 77], 16, 1, 128, 16, BF16, {}),
    "decode_group_40": ([1, 1], [200, 77], 40, 1, 64, 16, BF16, {}),
    "decode_mha": ([1, 1], [200, 77], 3, 3, 128, 16, BF16, {}),
    "drafts": ([3, 1, 4, 2], [50, 1, 4, 130], 8, 4, 128, 16, BF16, {}),
    "more_queries_than_keys": ([5, 3], [2, 3], 4, 2, 128, 16, F32, {}),
    "prompt": ([70, 1, 130], [70, 1, 130], 4, 2, 128, 16, BF16, {}),
    "prompt_64": ([200], [200], 2, 1, 64, 64, BF16, {}),
    "prompt_f32": ([65, 33], [65, 33], 2, 1, 128, 16, F32, {}),
    "prompt_256": ([70], [70], 3, 1, 256, 16, BF16, {}),
    "chunk": ([40, 64, 1], [300, 64, 257], 8, 2, 128, 32, BF16, {}),
    "cross": ([50, 3], [77, 200], 4, 2, 128, 16, BF16, dict(causal=False)),
    "cross_decode": ([1, 1], [77, 0], 4, 2, 64, 16, F32, dict(causal=False)),
    "window": ([1, 60, 2], [300, 200, 9], 4, 2, 128, 16, BF16, dict(window=33)),
    "window_1": ([4], [100], 4, 4, 128, 16, BF16, dict(window=1)),
    "window_f32": ([30, 1], [500, 130], 2, 2, 64, 16, F32, dict(window=128)),
    "plain_domain": ([1, 20], [90, 40], 4, 1, 128, 16, BF16, dict(unrotate=False)),
    "to_f32": ([1, 20], [90, 40], 4, 1, 128, 16, BF16, dict(out_dtype=F32)),
    "to_bf16": ([1, 20], [90, 40], 4, 1, 128, 16, F32, dict(out_dtype=BF16)),
    "nhd": ([1, 20], [90, 40], 4, 2, 128, 16, BF16, dict(layout="nhd")),
    "nhd_256": ([1, 20], [90, 40], 4, 2, 256, 16, F32, dict(layout="nhd")),
    "scale": ([2, 20], [90, 40], 4, 2, 64, 1024, BF16, dict(scale=-0.3)),
    "sharp": ([1, 20], [400, 40], 4, 2, 128, 16, BF16, dict(q_scale=30.0)),
    "padding": ([2, 20], [90, 40], 4, 2, 128, 16, BF16, dict(pad_rows=9)),
    "padding_decode": ([1, 1], [90, 40], 4, 2, 128, 16, BF16, dict(pad_rows=3)),
    "no_hint": ([1, 2], [90, 40], 4, 2, 128, 16, BF16, dict(hint=False)),
}


@pytest.mark.parametrize("name", ATT_CASES)
def test_attention_matches_oracle(name):
    *args, kw = ATT_CASES[name]
    _attend(len(name), *args, **kw)


def test_attention_many_requests():
    rng = np.random.default_rng(5)
    kv = rng.integers(0, 90, 150).tolist()
    _attend(6, [1] * 150, kv, 2, 1, 128, 16, BF16)
    _attend(7, rng.integers(0, 3, 150).tolist(), kv, 2, 1, 64, 16, F32)


def test_attention_hides_bad_pages_and_clamps_bad_lengths():
    rng = np.random.default_rng(8)
    D, page, pages = 128, 16, 6
    ck, sk = ku.pool(rng, pages, 1, page, D)
    cv, sv = ku.pool(rng, pages, 1, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = np.array([[0, -1, 2, 9], [3, 4, 5, 1]], np.int32)
    q = ku.dev(rng.standard_normal((3, 2, D)).astype(np.float32))
    for hint in (1, 40):
        got = ku.np64(rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array([60, 10 ** 9], np.int32)),
                                       ku.dev(np.array([0, 1, 2], np.int32)), max_q_len=hint, out=torch.zeros_like(q)))
        want, _, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, [60, 64], [0, 1, 2],
                                                D ** -0.5, True, 0, True)
        ku.close(got[:2], want[:2], ku.attention_tolerance(want, reach, size, F32, D, 64)[:2], "out")
    # starts outside the tokens or falling: no row out of bounds is touched, untouched rows stay
    out = torch.full_like(q, 5.0)
    rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array([-4, 10], np.int32)),
                     ku.dev(np.array([-7, -7, 1000], np.int32)), max_q_len=1, out=out)
    rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array([4, 10], np.int32)),
                     ku.dev(np.array([2, 1, 0], np.int32)), max_q_len=1, out=torch.full_like(q, 5.0))
    torch.cuda.synchronize()


def test_attention_nan_stays_in_its_row():
    # a NaN scale among a request's keys reaches the rows that see that key alone
    rng = np.random.default_rng(9)
    D, page = 128, 16
    for q_len in (4, 40):
        ck, sk = ku.pool(rng, 4, 1, page, D)
        cv, sv = ku.pool(rng, 4, 1, page, D)
        clean = ku.cache_of(ck, sk, cv, sv)
        sk2, sv2 = sk.copy(), sv.copy()
        sk2[2, 0, 8], sv2[2, 0, 8] = np.nan, np.inf  # key 40 of 3 * 16
        hurt = ku.cache_of(ck, sk2, cv, sv2)
        table, kv, cu = ku.dev(np.array([[0, 1, 2]], np.int32)), ku.dev(np.array([42], np.int32)), None
        cu = ku.dev(np.array([0, q_len], np.int32))
        q = ku.dev(rng.standard_normal((q_len, 2, D)).astype(np.float32), BF16)
        x = rw4.kv_attention(q, clean, table, kv, cu, max_q_len=q_len)
        y = rw4.kv_attention(q, hurt, table, kv, cu, max_q_len=q_len)
        assert torch.equal(x[:-2], y[:-2]) and torch.isnan(y[-2:]).all()
    q[3, 1, 5] = float("nan")
    y = rw4.kv_attention(q, clean, table, kv, cu, max_q_len=q_len)
    assert torch.isnan(y[3, 1]).all()
    y[3, 1] = x[3, 1]
    assert torch.equal(x, y)


def test_attention_reads_rows_written_by_quantize_act():
    # [slots, kv_heads * 128] rows of quantize_act (block and group 128) seen as pages
    rng = np.random.default_rng(10)
    hk, page, pages, D = 4, 32, 5, 128
    t = rw4.Transform.hadamard(hk * D, 128)
    rows = [ku.dev(rng.standard_normal((pages * page, hk * D)).astype(np.float32), BF16) for _ in range(2)]
    (qk, sk), (qv, sv) = (rw4.quantize_act(t, x) for x in rows)
    cache = rw4.KVCache.from_rows(qk, sk, qv, sv, page, hk)
    table, kv = np.array([[3, 1], [0, 4]], np.int32), [50, 33]
    q = ku.dev(rng.standard_normal((2, 8, D)).astype(np.float32), BF16)
    qr = rw4.qk_norm_rope(q, rotate=True)[0]
    got = rw4.kv_attention(qr, cache, ku.dev(table), ku.dev(np.array(kv, np.int32)),
                           ku.dev(np.array([0, 1, 2], np.int32)), max_q_len=1)
    want, _, reach, size = okv.kv_attention(
        ku.np64(qr), ku.opened(cache.k), ku.np64(cache.k_scale), ku.opened(cache.v), ku.np64(cache.v_scale), pages,
        table, kv, [0, 1, 2], D ** -0.5, True, 0, True)
    ku.close(ku.np64(got), want, ku.attention_tolerance(want, reach, size, BF16, D, 50), "out")


# ---------------------------------------------------------------- a run of them
class _Layer:
    """A decoder layer's attention part on W4A4 weights and an INT4 cache, with buffers for `tokens` tokens."""

    def __init__(self, tokens, B, pages, page, width, hq=4, hk=2, D=128, K=512):
        rng = np.random.default_rng(11)
        self.dims = (hq, hk, D, K)
        self.t = rw4.Transform.hadamard(K, 128)
        n = (hq + 2 * hk) * D
        self.qkv_w = rw4.pack_weight(self.t, ku.dev(rng.standard_normal((K, n)).astype(np.float32) * K ** -0.5))
        self.o_w = rw4.pack_weight(rw4.Transform.hadamard(hq * D, 128),
                                   ku.dev(rng.standard_normal((hq * D, K)).astype(np.float32) * K ** -0.5))
        self.wq, self.wk = (ku.dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
        self.rope = rw4.rope_table(4096, D)
        self.cache = rw4.KVCache.empty(pages, page, hk, D)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=ku.DEV)
        self.ring = torch.arange(pages, dtype=torch.int32, device=ku.DEV)
        self.state = torch.tensor([0, pages], dtype=torch.int32, device=ku.DEV)
        self.kv = torch.zeros(B, dtype=torch.int32, device=ku.DEV)
        self.page, self.tokens = page, tokens

    def step(self, x, new, most):
        hq, hk, D, K = self.dims
        T = x.shape[0]
        s = rw4.kv_slots(self.kv, new, self.table, self.ring, self.state, self.page, T, kv_len=self.kv,
                         free_state_out=self.state)
        y = rw4.w4a4_gemm(*rw4.quantize_act(self.t, x), *self.qkv_w).view(T, hq + 2 * hk, D)
        q = rw4.kv_append(self.cache, y[:, hq:hq + hk], y[:, hq + hk:], s.slot_map, y[:, :hq], self.wq, self.wk,
                          self.rope, s.positions)
        o = rw4.kv_attention(q, self.cache, self.table, self.kv, s.cu_new, max_q_len=most,
                             out=torch.zeros_like(q))
        z = rw4.w4a4_gemm(*rw4.quantize_act(rw4.Transform.hadamard(hq * D, 128), o.view(T, hq * D)), *self.o_w)
        return y, o, z, s


def _x(seed, T, K=512):
    return ku.dev(np.random.default_rng(seed).standard_normal((T, K)).astype(np.float32), BF16)


def test_serving_run_matches_oracle():
    # prompts of three requests, decode steps, one finishes and another arrives in its pages
    layer = _Layer(64, B=3, pages=9, page=16, width=6)
    hq, hk, D, _ = layer.dims
    past = [[], [], []]  # the qkv rows of each request so far
    steps = [[20, 33, 1], [1, 1, 1], [1, -1, 1], [4, 40, 1], [1, 1, 1]]
    for n, new in enumerate(steps):
        total = sum(max(x, 0) for x in new)
        T = total + 2
        y, o, z, s = layer.step(_x(n, T), ku.dev(np.array(new, np.int32)), max(new))
        assert s.served.tolist() == [1, 1, 1]
        y = ku.np64(y)
        at = 0
        for b, add in enumerate(new):
            past[b] = [] if add < 0 else past[b] + [y[at + i] for i in range(add)]
            at += max(add, 0)
        assert layer.kv.tolist() == [len(p) for p in past]
        got, at = ku.np64(o), 0
        cs = ku.np64(layer.rope)
        wq, wk = ku.np64(layer.wq), ku.np64(layer.wk)
        for b, add in enumerate(new):
            if add <= 0:
                continue
            rows = np.stack(past[b])
            L = len(rows)
            pos = np.arange(L)
            zk, fk = okv.norm_rope(rows[:, hq:hq + hk], wk, 1e-6, cs, pos, False)
            ck, sk = okv.quantize_heads(zk, fk, True)
            cv, sv = okv.quantize_heads(rows[:, hq + hk:], np.ones((L, hk, 1)), True)
            zq, fq = okv.norm_rope(rows[L - add:, :hq], wq, 1e-6, cs, pos[L - add:], False)
            q = okv.rotate_heads(zq * fq)
            qb = ku.np64(ku.dev(q.astype(np.float32), BF16))
            P = 16
            pages = -(-L // P)

            def paged(a):
                a = np.concatenate([a, np.zeros((pages * P - L,) + a.shape[1:], a.dtype)])
                return np.moveaxis(a.reshape((pages, P) + a.shape[1:]), 1, 2)

            want, _, reach, size = okv.kv_attention(qb, paged(ck), paged(sk), paged(cv), paged(sv), pages,
                                                    np.arange(pages)[None], [L], [0, add], D ** -0.5, True, 0, True)
            # the queries may round to the neighbouring bf16 where the two evaluations straddle a border: one
            # step of 2 half_step in one of D products at most enters a score
            tol = ku.attention_tolerance(want, reach, size, BF16, D, L) + (
                4 * ku.half_step(BF16) * size * reach)[..., None]
            ku.close(got[at:at + add], want, tol, f"step {n} request {b}")
            at += add
        assert (got[total:] == 0).all()


def test_captured_decode_step_replays():
    # the whole step in one graph: lengths, tables and the free list move on the device; each replay equals the
    # eager layer's step on the same input
    B, steps = 3, 6
    eager, graphed = (_Layer(B, B=B, pages=12, page=16, width=6) for _ in range(2))
    first = np.array([14, 30, 1], np.int32)
    for layer in (eager, graphed):
        layer.step(_x(50, int(first.sum())), ku.dev(first), 30)
    one = ku.dev(np.ones(B, np.int32))
    x = _x(51, B)
    keep = [t.clone() for t in (graphed.kv, graphed.state, graphed.table, graphed.ring)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(x, one, 1)
    torch.cuda.current_stream().wait_stream(side)
    for t, o in zip((graphed.kv, graphed.state, graphed.table, graphed.ring), keep):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, o, z, s = graphed.step(x, one, 1)
    for n in range(steps):
        x.copy_(_x(60 + n, B))
        g.replay()
        junk = torch.randn(1000, device=ku.DEV).sum()  # unrelated eager work between replays
        torch.cuda.synchronize()
        _, eo, ez, es = eager.step(x, one, 1)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(z, ez) and torch.equal(s.slot_map, es.slot_map)
        assert torch.equal(graphed.kv, eager.kv) and torch.equal(graphed.state, eager.state)
        assert torch.isfinite(junk)
    assert torch.equal(graphed.cache.k, eager.cache.k) and torch.equal(graphed.table, eager.table)


def test_prepared_calls_and_streams():
    rng = np.random.default_rng(12)
    D, page = 128, 16
    ck, sk = ku.pool(rng, 20, 2, page, D)
    cv, sv = ku.pool(rng, 20, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = ku.dev(rng.permutation(20).reshape(2, 10).astype(np.int32))
    kv, cu = ku.dev(np.array([150, 160], np.int32)), ku.dev(np.array([0, 1, 2], np.int32))
    q = [ku.dev(rng.standard_normal((2, 8, D)).astype(np.float32), BF16) for _ in range(2)]
    want = [rw4.kv_attention(x, cache, table, kv, cu, max_q_len=1) for x in q]
    calls = [rw4.prepare_kv_attention(x, cache, table, kv, cu, max_q_len=1) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):  # two calls at once, a workspace each
        for c, st in zip(calls, streams):
            with torch.cuda.stream(st):
                got = c()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c.result, w)
    assert got is calls[1].result


def test_slots_without_requests():
    e = torch.empty(0, dtype=torch.int32, device=ku.DEV)
    state = ku.dev(np.array([3, 4], np.int32))
    got = rw4.kv_slots(e, e, torch.empty((0, 5), dtype=torch.int32, device=ku.DEV), ku.dev(np.arange(8, dtype=np.int32)),
                       state, 16, 7)
    torch.cuda.synchronize()
    assert got.cu_new.tolist() == [0] and got.free_state.tolist() == [3, 4]
    assert got.slot_map.tolist() == [-1] * 7 and got.positions.tolist() == [-1] * 7


def test_captured_chunk_replays():
    # the kernel for many rows under capture; lengths change between the replays
    rng = np.random.default_rng(13)
    D, page = 64, 16
    ck, sk = ku.pool(rng, 80, 2, page, D)
    cv, sv = ku.pool(rng, 80, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = ku.dev(rng.permutation(80).reshape(2, 40).astype(np.int32))
    kv, cu = ku.dev(np.array([500, 640], np.int32)), ku.dev(np.array([0, 70, 150], np.int32))
    q = ku.dev(rng.standard_normal((150, 8, D)).astype(np.float32), BF16)
    out = torch.zeros_like(q)
    args = dict(max_q_len=80, out=out, workspace=torch.empty(
        rw4.kv_attention_workspace_bytes(150, 2, 8, 2, D), dtype=torch.uint8, device=ku.DEV))
    rw4.kv_attention(q, cache, table, kv, cu, **args)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        rw4.kv_attention(q, cache, table, kv, cu, **args)
    for lens in ([500, 640], [90, 80], [640, 81], [1, 333]):
        kv.copy_(ku.dev(np.array(lens, np.int32)))
        out.fill_(9.0)
        g.replay()
        junk = torch.randn(1000, device=ku.DEV).sum()
        torch.cuda.synchronize()
        want = rw4.kv_attention(q, cache, table, kv, cu, max_q_len=80)
        assert torch.equal(out, want) and torch.isfinite(junk)


def test_cache_beyond_32_bit_offsets():
    # pages of 32 KiB up to byte 5.4e9 of each half; the same rows in a small cache give the same bits
    D, hk, page, pages = 128, 8, 64, 165000
    cache = rw4.KVCache(*(torch.empty(s, dtype=d, device=ku.DEV) for s, d in
                          (((pages, hk, page, D // 2), torch.uint8),) * 2 + (((pages, hk, page), F32),) * 2))
    small = rw4.KVCache.empty(4, page, hk, D)
    T = 150
    k, v, q = _rows(1, T, hk, D, BF16), _rows(2, T, hk, D, BF16), _rows(3, T, 16, D, BF16)
    high = np.array([[pages - 1, 131072, 164001]], np.int32)
    for c, ids in ((cache, high), (small, np.array([[2, 0, 3]], np.int32))):
        j = np.arange(T)
        rw4.kv_append(c, k, v, ku.dev(ids[0, j // page].astype(np.int64) * page + j % page))
    kv, cu = ku.dev(np.array([T], np.int32)), ku.dev(np.array([0, T], np.int32))
    for rows, hint in ((T, T), (1, 1)):
        cu = ku.dev(np.array([0, rows], np.int32))
        got = rw4.kv_attention(q[:rows], cache, ku.dev(high), kv, cu, max_q_len=hint)
        want = rw4.kv_attention(q[:rows], small, ku.dev(np.array([[2, 0, 3]], np.int32)), kv, cu, max_q_len=hint)
        assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32), (128, F32)])
def test_attention_large_batches_match_a_row_at_a_time(D, dtype):
    # many units (whole ones, cut ones) against single-request calls on the same cache
    rng = np.random.default_rng(14)
    hk, group, page, B = 2, 4, 16, 24
    q_lens = rng.integers(0, 260, B).tolist()
    kv_lens = [int(n + rng.integers(0, 900)) for n in q_lens]
    pages = sum(-(-n // page) for n in kv_lens) + 1
    table = ku.page_table(rng, kv_lens, page, max(-(-n // page) for n in kv_lens), pages)
    ck, sk = ku.pool(rng, pages, hk, page, D)
    cv, sv = ku.pool(rng, pages, hk, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = ku.dev(rng.standard_normal((int(cu[-1]), hk * group, D)).astype(np.float32), dtype)
    td, kd = ku.dev(table), ku.dev(np.array(kv_lens, np.int32))
    full, lse = rw4.kv_attention(q, cache, td, kd, ku.dev(cu), max_q_len=260, return_lse=True)
    few, lse2 = rw4.kv_attention(q, cache, td, kd, ku.dev(cu), max_q_len=1, return_lse=True)  # the other kernel
    # what a relative error of the probabilities acts on: sum_j p_j |v_j|, from the magnitudes of the values; twice
    # the tolerance against the definition, since both sides have it, and 1 % for the bound's own rounding
    mags = rw4.kv_attention(q, ku.cache_of(ck, sk, np.abs(cv), sv), td, kd, ku.dev(cu), max_q_len=1, unrotate=False,
                            out_dtype=F32)
    reach = 1.01 * ku.np64(mags).sum(-1) / D ** 0.5
    size = D ** -0.5 * 7 * float(sk.max()) * ku.np64(q.float().abs().sum(-1))
    tol = 2 * ku.attention_tolerance(ku.np64(few), reach, size, dtype, D, max(kv_lens))
    ku.close(ku.np64(full), ku.np64(few), tol, "kernels")
    lt = 2 * ((D + 8) * ku.U24 * size + (64 + max(kv_lens)) * ku.U24 + 4 * ku.U24 * np.abs(ku.np64(lse)))
    ku.close(ku.np64(lse), ku.np64(lse2), lt, "lse")
    for b in (0, 5, 11, 23):
        a0, a1 = int(cu[b]), int(cu[b + 1])
        if a0 < a1:
            one = rw4.kv_attention(q[a0:a1], cache, td[b:b + 1].contiguous(), kd[b:b + 1],
                                   ku.dev(np.array([0, a1 - a0], np.int32)))
            ku.close(ku.np64(one), ku.np64(full)[a0:a1], tol[a0:a1], f"request {b}")


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (128, F32)])
def test_attention_many_rows_hide_bad_pages_and_clamp_bad_lengths(D, dtype):
    # pages out of range in the middle of steps and as whole steps; a length beyond the table
    rng = np.random.default_rng(17)
    page, pages, lens, q_lens = 16, 24, [190, 10 ** 9], [70, 80]
    ck, sk = ku.pool(rng, pages, 2, page, D)
    cv, sv = ku.pool(rng, pages, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    table = rng.permutation(pages).reshape(2, 12).astype(np.int32)
    table[0, 1], table[0, 4:8] = -1, (pages, -2 ** 31, 2 ** 31 - 1, pages + 3)
    table[1, 0], table[1, 11] = -5, pages
    cu = np.array([0, 70, 150], np.int32)
    q = ku.dev((1.5 * rng.standard_normal((150, 4, D))).astype(np.float32), dtype)
    out, lse = rw4.kv_attention(q, cache, ku.dev(table), ku.dev(np.array(lens, np.int32)), ku.dev(cu),
                                max_q_len=max(q_lens), return_lse=True)
    kv = [190, 12 * page]
    want, wl, reach, size = okv.kv_attention(ku.np64(q), ck, sk, cv, sv, pages, table, kv, cu, D ** -0.5, True, 0, True)
    ku.close(ku.np64(out), want, ku.attention_tolerance(want, reach, size, dtype, D, 192), "out")
    lt = (D + 8) * ku.U24 * size + (64 + 192) * ku.U24 + 4 * ku.U24 * np.abs(wl)
    ku.close(ku.np64(lse), wl, lt, "lse")


def test_attention_cut_units_behind_a_long_padding():
    # tokens for far more units than the requests have: units are cut all the same, and merged by few blocks
    rng = np.random.default_rng(23)
    D, page, kv_lens, q_lens, padded = 128, 64, [6000, 5801], [60, 75], 17000
    pages = sum(-(-n // page) for n in kv_lens)
    table = ku.dev(ku.page_table(rng, kv_lens, page, -(-6000 // page), pages))
    ck, sk = ku.pool(rng, pages, 2, page, D)
    cv, sv = ku.pool(rng, pages, 2, page, D)
    cache = ku.cache_of(ck, sk, cv, sv)
    kv, cu, n = ku.dev(np.array(kv_lens, np.int32)), ku.dev(np.array([0, 60, 135], np.int32)), 135
    q = torch.zeros((padded, 8, D), dtype=BF16, device=ku.DEV)
    q[:n] = ku.dev(rng.standard_normal((n, 8, D)).astype(np.float32), BF16)
    out = torch.full_like(q, 3.0)
    _, lse = rw4.kv_attention(q, cache, table, kv, cu, max_q_len=75, out=out, return_lse=True)
    want, wl = rw4.kv_attention(q[:n], cache, table, kv, cu, max_q_len=75, return_lse=True)
    assert torch.equal(out[:n], want) and torch.equal(lse[:n], wl)
    assert (out[n:] == 3.0).all()
    for b, (a0, a1) in enumerate(((0, 60), (60, 135))):  # and alone, against the oracle
        o, _, reach, size = okv.kv_attention(ku.np64(q[a0:a1]), ck, sk, cv, sv, pages, table[b:b + 1].cpu().numpy(),
                                             kv_lens[b:b + 1], [0, a1 - a0], D ** -0.5, True, 0, True)
        tol = ku.attention_tolerance(o, reach, size, BF16, D, kv_lens[b])
        ku.close(ku.np64(out[a0:a1]), o, tol, f"request {b}")
